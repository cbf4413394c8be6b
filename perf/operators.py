"""The key/value cache operators: cases to measure, their plain forms, and their values in 64 bits.

A cache holds the keys and values of B sequences in pages of `page` tokens, pages
[n_pages, Hk, page, d], found through a table [B, max_pages]; `length` [B] tokens of each
sequence are valid. Per page it keeps the sum of its keys (`ksum`), per slot the attention
weight the slot has received (`mass`) and its token's position (`pos`). Hq = G * Hk query
heads share the Hk key heads in groups of G. Operators:

  append  write the keys and values of new tokens into the pages, with their sums
  score   a cheap score of every page for every query: softmax over the pages' mean keys
  attn    attention of T new tokens (a drafted tree, or one token) over the cache, whole or
          the pages of a plan, and over each other where the tree's mask allows
  mass    add the attention weight that each slot received to `mass`
  evict   keep the `budget` slots with the largest mass (the last ones always), compacted

Every case is shaped from: op, B sequences, Hq and Hk heads, d, page, type, T new tokens,
and lengths spread evenly from len_min to len_max over the sequences.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, B, Hq, Hk, d, page, type, len_min, len_max, T=1, budget=0, weighted=False,
          per_token=True):
    c = dict(op=op, B=B, Hq=Hq, Hk=Hk, d=d, page=page, type=type, len_min=len_min,
             len_max=len_max, T=T, budget=budget, weighted=weighted, per_token=per_token)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # the key and value of one new token for each of 32 sequences, every step of a serving loop
        _case("append_token", "append", 32, 40, 8, 128, 64, "bf16", 900, 32760),
        # a prompt of 32760 tokens in a batch of two, written at once
        _case("append_prompt", "append", 2, 12, 12, 128, 128, "bf16", 0, 37, T=32760),
        # scoring the pages of one long sequence for the next token, its first and last pages
        # always kept: a latency-bound call
        _case("score_token", "score", 1, 24, 8, 128, 128, "bf16", 262144, 262144,
              weighted=True),
        # scoring a ragged batch with small pages
        _case("score_batch", "score", 32, 40, 8, 128, 16, "bf16", 4097, 32760),
        # the first tokens after a short prompt: the smallest call
        _case("attn_token_short", "attn", 1, 12, 12, 64, 16, "fp16", 1000, 1000),
        # one token of each sequence of a ragged batch: the ordinary serving step
        _case("attn_token_batch", "attn", 16, 40, 8, 128, 64, "bf16", 1023, 32760),
        # a tree of 64 drafted tokens verified against the cache
        _case("attn_tree", "attn", 8, 40, 8, 128, 128, "bf16", 16001, 32760, T=64),
        # one token over a tenth of the pages, sampled with weights, of four long sequences
        _case("attn_token_selected", "attn", 4, 24, 8, 128, 128, "bf16", 60000, 118800,
              budget=93, weighted=True),
        # the weight one token per sequence gave to every slot
        _case("mass_token", "mass", 16, 40, 8, 128, 64, "bf16", 1023, 32760),
        # the weights of a prompt's last 64 tokens, as a prompt's eviction wants them
        _case("mass_window", "mass", 2, 24, 8, 128, 128, "bf16", 60000, 118800, T=64),
        # eviction in a running loop: a page's worth over the budget
        _case("evict_step", "evict", 32, 40, 8, 128, 64, "bf16", 4096, 4160, budget=4096),
        # eviction after a long prompt: a tenth stays
        _case("evict_prompt", "evict", 4, 24, 8, 128, 128, "bf16", 60000, 118800, budget=11880),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "score", "attn", "attn", "attn", "mass", "evict"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    type = rng.choice(["bf16", "fp16"])
    Hk = rng.choice([1, 2, 3, 4, 8, 12])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    B = log(1, 32)
    # the whole cache stays under 2 GB, keys and values
    most = min(262144, (1 << 30) // (B * Hk * d * 2))
    len_max = log(min(500, most), most)
    len_min = rng.choice([len_max, log(1, len_max)])
    T, budget, weighted, per_token = 1, 0, False, True
    if op == "append":
        T = rng.choice([1, log(1, 64), log(64, 4096)])
    elif op == "score":
        T = rng.choice([1, 1, log(2, 32)])
        weighted, per_token = rng.random() < 0.5, rng.random() < 0.5
    elif op == "attn":
        T = rng.choice([1, log(2, 16), log(16, 128)])
        # the plain form's scores stay within those of the largest listed case
        T = max(1, min(T, 600_000_000 // (B * Hk * G * len_max)))
        pages = -(-len_max // page)
        if rng.random() < 0.5:
            budget, weighted = max(1, pages * log(5, 30) // 100), rng.random() < 0.5
            per_token = T <= 16 and rng.random() < 0.5
    elif op == "mass":
        T = rng.choice([1, log(2, 128)])
        T = max(1, min(T, len_max, 300_000_000 // (B * Hk * G * len_max)))
    else:
        budget = log(max(1, len_max // 20), len_max)
    return _case(None, op, B, Hk * G, Hk, d, page, type, len_min, len_max, T, budget, weighted,
                 per_token)


def _lengths(c):
    B, lo, hi = c["B"], c["len_min"], c["len_max"]
    return [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]


def _counts(c):
    """New tokens of each sequence: all T for the first, down to half of T for the last."""
    B, T = c["B"], c["T"]
    if c["op"] == "mass":
        return [min(n, T - (T // 2) * b // max(1, B - 1)) for b, n in enumerate(_lengths(c))]
    return [T - (T // 2) * b // max(1, B - 1) for b in range(B)]


def _always(c):
    """score: the first and last pages that are always kept, which score 2."""
    return (1, 2) if c["weighted"] else (0, 0)


def _max_pages(c):
    page = c["page"]
    room = c["len_max"] + (c["T"] if c["op"] == "append" else 0)
    # a page more than needed, and every page allocated: no write of a plain form collides
    return -(-max(room, c["budget"] if c["op"] == "evict" else 0) // page) + 2


def work(case):
    c = case
    B, Hq, Hk, d, page, T = (c[k] for k in ("B", "Hq", "Hk", "d", "page", "T"))
    L, n = _lengths(c), _counts(c)
    rows = sum(n)
    if c["op"] == "append":
        touched = sum((l + t - 1) // page - l // page + 1 for l, t in zip(L, n))
        old = sum(l % page for l in L)  # keys of the open page, which its sum reads again
        return {"bytes": Hk * (rows * d * 2 * 4 + rows * 8 + old * d * 2 + touched * d * 4),
                "flops": Hk * (rows + old) * d}
    if c["op"] == "score":
        pages = sum(-(-l // page) for l in L)
        tp = T if c["per_token"] else 1
        return {"bytes": pages * Hk * d * 4 + rows * Hq * d * 2 + B * Hk * tp * _max_pages(c) * 4,
                "flops": sum(-(-l // page) * t for l, t in zip(L, n)) * Hq * (2 * d + 4)}
    if c["op"] == "attn":
        if c["budget"]:
            kept = [min(l, c["budget"] * page) for l in L]
            uniq = [min(l, k * (t if c["per_token"] else 1)) for l, k, t in zip(L, kept, n)]
        else:
            kept = uniq = L
        return {"bytes": (sum(uniq) + rows) * Hk * d * 4 + rows * Hq * (d * 4 + 4),
                "flops": sum((k + t) * t for k, t in zip(kept, n)) * Hq * (4 * d + 5)}
    if c["op"] == "mass":
        return {"bytes": sum(L) * Hk * (d * 2 + 8) + rows * Hq * (d * 2 + 4),
                "flops": sum(l * t for l, t in zip(L, n)) * Hq * (2 * d + 4)}
    keep = [min(l, c["budget"]) for l in L]
    # survivors behind the budget move: about the share of the slots that stays
    moved = sum(k * (l - k) // max(1, l) for l, k in zip(L, keep))
    return {"bytes": Hk * (sum(L) * 8 + moved * (d * 8 + 16) + sum(keep) * 4),
            "flops": Hk * sum(L) * 4}


def prepare(case, seed):
    c = case
    B, Hq, Hk, d, page, T = (c[k] for k in ("B", "Hq", "Hk", "d", "page", "T"))
    op, dev, dtype = c["op"], "cuda", _TYPES[c["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=dtype):
        x = torch.empty(shape, device=dev, dtype=dtype)
        return x.normal_(0.0, scale, generator=g)

    mp = _max_pages(c)
    n_pages = B * mp
    L = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
    n = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
    st = dict(case=c, length=L.clone(), len0=L, n=n)
    st["table"] = torch.randperm(n_pages, generator=g, device=dev).int().view(B, mp)
    if op != "score":
        # keys with a common direction per head, so that some slots weigh much more than others
        k = randn(n_pages, Hk, page, d)
        u = randn(1, Hk, 1, d, dtype=torch.float32)
        u = u / u.norm(dim=-1, keepdim=True)
        gain = randn(n_pages, Hk, page, 1, dtype=torch.float32) * 2.0
        k += (gain * u).to(dtype)
        st["k"] = k
        st["u"] = u.view(Hk, d)
    else:  # scoring reads the sums alone: the pages' own contents do not matter to it
        st["k"] = torch.zeros(n_pages, Hk, page, d, device=dev, dtype=dtype)
    if op in ("append", "attn", "evict"):
        st["v"] = randn(n_pages, Hk, page, d)
    if op in ("append", "score", "evict"):
        st["ksum"] = randn(n_pages, Hk, d, scale=0.5 * page, dtype=torch.float32)
    if op in ("append", "mass", "evict"):
        # heavy-tailed: a few slots hold most of the weight
        st["mass"] = randn(n_pages, Hk, page, dtype=torch.float32).mul_(2.0).exp_()
    slot = torch.arange(mp * page, device=dev, dtype=torch.int32)
    if op in ("append", "evict"):
        # positions run ahead of slots where earlier evictions dropped tokens
        pos = (slot * 2).view(1, mp, 1, page).expand(B, mp, Hk, page)
        st["pos"] = torch.empty(n_pages, Hk, page, device=dev, dtype=torch.int32)
        st["pos"][st["table"].long()] = pos
    if op in ("score", "attn", "mass"):
        st["q"] = randn(B, Hq, T, d)
        if op != "score":
            q = st["q"].view(B, Hk, Hq // Hk, T, d)
            q += (st["u"] * math.sqrt(d)).to(dtype).view(1, Hk, 1, 1, d)
    if op in ("append", "attn"):
        st["k_new"], st["v_new"] = randn(B, Hk, T, d), randn(B, Hk, T, d)
    if op == "append":
        st["start"], st["pos0"] = L, L * 2
        # the accepted tokens' places among the drafted ones, ascending
        keep = torch.rand(B, T, generator=g, device=dev).argsort(dim=1)
        i = torch.arange(T, device=dev)
        keep = torch.where(i < n.view(B, 1), keep, T + i)
        st["sel"] = keep.sort(dim=1).values.clamp_(max=T - 1).int()
    if op == "attn" and T > 1:
        # a random tree: token i's parent is one of the tokens before it (-1: the context)
        r = torch.rand(B, T, generator=g, device=dev)
        i = torch.arange(T, device=dev)
        parent = (r * (i + 1)).long() - 1
        tree = torch.zeros(B, T, T, dtype=torch.bool, device=dev)
        for t in range(T):
            p = parent[:, t]
            tree[:, t] = tree[torch.arange(B, device=dev), p.clamp(min=0)] & (p >= 0).view(B, 1)
            tree[:, t, t] = True
        st["tree"] = tree
    if op == "attn" and c["budget"]:
        tp = T if c["per_token"] else 1
        pages = (L + page - 1) // page
        ids = torch.arange(mp, device=dev)
        r = torch.rand(B, Hk, tp, mp, generator=g, device=dev)
        r = torch.where(ids < pages.view(B, 1, 1, 1), r, 2.0)
        kept = r.argsort(dim=-1)[..., : c["budget"]]
        cnt = torch.clamp(pages, max=c["budget"]).view(B, 1, 1).expand(B, Hk, tp)
        i = torch.arange(c["budget"], device=dev)
        kept = torch.where(i < cnt.unsqueeze(-1), kept, mp).sort(dim=-1).values
        idx = torch.full((B, Hk, tp, mp), -1, device=dev, dtype=torch.int32)
        idx[..., : kept.shape[-1]] = torch.where(kept < mp, kept, -1).int()
        st["idx"], st["cnt"] = idx, cnt.contiguous().int()
        if c["weighted"]:  # one over an inclusion probability
            w = 1.0 / torch.rand(idx.shape, generator=g, device=dev).clamp_(min=0.05)
            st["w"] = torch.where(idx >= 0, w, 0.0)
    if op == "mass":
        # row i's log of the sum over what it sees, as the attention returned it
        s = _logits(st)
        st["lse"] = torch.logsumexp(s, dim=-1)
        st["lse"] = torch.where(_rows(st), st["lse"], 0.0).contiguous()
        st["out"] = torch.zeros_like(st["mass"])
    if op == "evict":
        st["mass0"], st["pos0"] = st["mass"].clone(), st["pos"].clone()
        st["next_pos"] = L * 2
    return st


# --------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------


def _gathered(pages, table):
    """[n_pages, Hk, page, ...] through [B, max_pages] as [B, Hk, max_pages * page, ...]."""
    x = pages[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _rows(st):
    """Valid query rows, [B, 1, T]."""
    T = st["case"]["T"]
    return (torch.arange(T, device="cuda") < st["n"].view(-1, 1)).unsqueeze(1)


def _logits(st):
    """mass: the logits of row i of each sequence over the slots it sees, else -inf."""
    c = st["case"]
    B, Hq, Hk, d, T = (c[k] for k in ("B", "Hq", "Hk", "d", "T"))
    k = _gathered(st["k"], st["table"]).float()
    q = st["q"].float().view(B, Hk, Hq // Hk * T, d)
    s = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).view(B, Hq, T, -1)
    slot = torch.arange(s.shape[-1], device="cuda")
    i = torch.arange(T, device="cuda").view(1, T, 1)
    sees = slot < (st["len0"] - st["n"]).view(B, 1, 1) + i + 1
    sees &= i < st["n"].view(B, 1, 1)
    return s.masked_fill_(~sees.unsqueeze(1), -math.inf)


def _append(st):
    c = st["case"]
    B, T, page = c["B"], c["T"], c["page"]
    k, v, mass, pos, ksum, table = (st[x] for x in ("k", "v", "mass", "pos", "ksum", "table"))
    table = table.long()
    i = torch.arange(T, device="cuda", dtype=torch.int32).view(1, T)
    new = (i < st["n"].view(B, 1)).unsqueeze(-1)  # [B, T, 1]
    slot = (st["start"].view(B, 1) + i).long()
    pg, off = table.gather(1, slot // page), slot % page
    sel = st["sel"].long().unsqueeze(1).unsqueeze(-1).expand(-1, c["Hk"], -1, c["d"])
    k_new, v_new = (x.gather(2, sel).transpose(1, 2) for x in (st["k_new"], st["v_new"]))
    k[pg, :, off] = torch.where(new.unsqueeze(-1), k_new, k[pg, :, off])
    v[pg, :, off] = torch.where(new.unsqueeze(-1), v_new, v[pg, :, off])
    mass[pg, :, off] = torch.where(new, 0.0, mass[pg, :, off])
    p = (st["pos0"].view(B, 1) + i).unsqueeze(-1)
    pos[pg, :, off] = torch.where(new, p, pos[pg, :, off])
    torch.add(st["start"], st["n"], out=st["length"])
    # the sums of the pages that got a token
    t = torch.arange((T - 1) // page + 2, device="cuda").view(1, -1)
    lp = (st["start"].view(B, 1) // page + t).long()
    pg = table.gather(1, lp)
    row = lp.unsqueeze(-1) * page + torch.arange(page, device="cuda")
    valid = (row < st["length"].view(B, 1, 1)).view(B, -1, 1, page, 1)
    total = torch.where(valid, k[pg].float(), 0.0).sum(dim=3)
    got = (lp * page < st["length"].view(B, 1)) & (st["n"].view(B, 1) > 0)
    ksum[pg] = torch.where(got.view(B, -1, 1, 1), total, ksum[pg])
    return [k, v, mass, pos, ksum, st["length"]]


def _score(st):
    c = st["case"]
    B, Hq, Hk, d, T, page = (c[k] for k in ("B", "Hq", "Hk", "d", "T", "page"))
    first, recent = _always(c)
    s = st["ksum"][st["table"].long()].transpose(1, 2)  # [B, Hk, mp, d]
    mp = s.shape[2]
    at = torch.arange(mp, device="cuda").view(1, mp)
    size = (st["len0"].view(B, 1) - at * page).clamp(0, page)
    mean = s / size.clamp(min=1).view(B, 1, mp, 1)
    q = st["q"].float().view(B, Hk, Hq // Hk * T, d)
    x = (q @ mean.transpose(-1, -2)).mul_(d ** -0.5)
    there = (size > 0).view(B, 1, 1, mp)
    x = x.masked_fill_(~there, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    p = p / p.sum(dim=-1, keepdim=True).clamp(min=1e-38)
    p = p.view(B, Hk, Hq // Hk, T, mp) * _rows(st).view(B, 1, 1, T, 1)
    p = p.sum(dim=2) / (Hq // Hk)
    rows = _rows(st).view(B, 1, T, 1)
    if not c["per_token"]:
        p = p.sum(dim=2, keepdim=True) / st["n"].clamp(min=1).view(B, 1, 1, 1)
        rows = rows.any(dim=2, keepdim=True)
    pages = (size > 0).sum(dim=1).view(B, 1)
    kept = ((at < first) | (at >= pages - recent)) & (at < pages)
    return torch.where(kept.view(B, 1, 1, mp) & rows, 2.0, p)


def _attn(st):
    c = st["case"]
    B, Hq, Hk, d, T, page = (c[k] for k in ("B", "Hq", "Hk", "d", "T", "page"))
    G = Hq // Hk
    k, v = (_gathered(st[x], st["table"]).float() for x in ("k", "v"))
    mp = st["table"].shape[1]
    k = torch.cat([k, st["k_new"].float()], dim=2)
    v = torch.cat([v, st["v_new"].float()], dim=2)
    q = st["q"].float().view(B, Hk, G * T, d)
    s = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).view(B, Hk, G, T, -1)
    slot = torch.arange(mp * page, device="cuda")
    ctx = (slot < st["len0"].view(B, 1)).view(B, 1, 1, -1)
    if "idx" in st:
        there = (torch.arange(mp, device="cuda") < st["cnt"].unsqueeze(-1))
        at = torch.where(there, st["idx"], mp).long()
        bias = torch.full((*at.shape[:3], mp + 1), -math.inf, device="cuda")
        bias.scatter_(-1, at, torch.log(st["w"]) if "w" in st else torch.zeros(at.shape, device="cuda"))
        bias = bias[..., :mp].repeat_interleave(page, dim=-1)
        bias = torch.where(ctx, bias, -math.inf)
    else:
        bias = torch.zeros(ctx.shape, device="cuda").masked_fill_(~ctx, -math.inf)
    s[..., : mp * page] += bias.unsqueeze(2)
    j = torch.arange(T, device="cuda")
    sees = (j < st["n"].view(B, 1)).view(B, 1, T) & (st["tree"] if "tree" in st else j.view(T, 1) >= j)
    s[..., mp * page :].masked_fill_(~sees.view(B, 1, 1, T, T), -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = (p.view(B, Hk, G * T, -1) @ v).view(B, Hq, T, d)
    l, m = l.view(B, Hq, T), m.view(B, Hq, T)
    rows = _rows(st)
    lse = torch.where(rows, m + torch.log(l), 0.0)
    o = torch.where((rows & (l > 0)).unsqueeze(-1), o / l.unsqueeze(-1), 0.0)
    return [o.to(st["q"].dtype), lse]


def _mass(st):
    c = st["case"]
    B, Hq, Hk, T = (c[k] for k in ("B", "Hq", "Hk", "T"))
    got = torch.exp(_logits(st).sub_(st["lse"].unsqueeze(-1))).view(B, Hk, Hq // Hk * T, -1).sum(dim=2)
    old = _gathered(st["mass"], st["table"])
    slot = torch.arange(old.shape[-1], device="cuda")
    there = (slot < st["len0"].view(B, 1)).view(B, 1, -1)
    new = torch.where(there, old + got, _gathered(st["out"], st["table"]))
    page, mp = c["page"], st["table"].shape[1]
    st["out"][st["table"].long()] = new.view(B, Hk, mp, page).transpose(1, 2)
    return st["out"]


def _evict(st):
    c = st["case"]
    B, Hk, page, n = c["B"], c["Hk"], c["page"], c["budget"]
    recent = min(64, n // 2)
    table, len0 = st["table"].long(), st["len0"].view(B, 1, 1)
    mp = table.shape[1]
    x = _gathered(st["mass0"], st["table"])
    pos = _gathered(st["pos0"], st["table"])
    slot = torch.arange(mp * page, device="cuda").view(1, 1, -1)
    x = torch.where(pos >= (st["next_pos"] - recent).view(B, 1, 1), math.inf, x)
    x = torch.where(slot < len0, x, -1.0)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    kept.scatter_(-1, order[..., :n], True)
    kept &= slot < len0
    # the k-th hole below the budget takes the k-th survivor behind it
    mover = torch.where(kept & (slot >= n), slot, mp * page).sort(dim=-1).values
    hole = ~kept[..., :n]
    rank = (hole.cumsum(dim=-1) - 1).clamp(min=0)
    src = torch.where(hole, mover.gather(-1, rank), slot[..., :n])
    src = torch.where(slot[..., :n] < len0, src, -1)
    count = torch.clamp(st["len0"], max=n)
    # move, each head for itself; a slot without a source keeps what it holds
    frm = torch.where(src < 0, slot[..., :n], src)
    to = slot[..., :n].expand_as(frm)
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    h = torch.arange(Hk, device="cuda").view(1, Hk, 1)
    fp, tp = table[b, frm // page], table[b, to // page]
    fo, to = frm % page, to % page
    k, v, mass, pos, ksum = (st[x] for x in ("k", "v", "mass", "pos", "ksum"))
    k[tp, h, to] = k[fp, h, fo]
    v[tp, h, to] = v[fp, h, fo]
    mass[tp, h, to] = mass[fp, h, fo]
    pos[tp, h, to] = pos[fp, h, fo]
    st["length"].copy_(count)
    # the sums of the pages that changed, and of the last page where it is not full
    np_ = -(-n // page)
    pad = np_ * page - n
    row = torch.arange(np_ * page, device="cuda").view(1, 1, np_, page)
    changed = torch.nn.functional.pad((src != slot[..., :n]) & (src >= 0), (0, pad)).view(B, Hk, np_, page).any(-1)
    last = (row[..., 0] <= (count.view(B, 1, 1) - 1)) & (row[..., -1] >= count.view(B, 1, 1))
    changed |= last
    pg = table[:, :np_]
    kp = k[pg].transpose(1, 2).float()  # [B, Hk, np_, page, d]
    total = torch.where((row < count.view(B, 1, 1, 1)).unsqueeze(-1), kp, 0.0).sum(dim=3)
    old = ksum[pg].transpose(1, 2)
    ksum[pg] = torch.where(changed.unsqueeze(-1), total, old).transpose(1, 2)
    return [src.int(), count, k, v, mass, pos, ksum, st["length"]]


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------


def _cache(st):
    """The program's cache handle over the state's tensors, made on the first pass."""
    if "cache" not in st:
        import block_sparse_attention_ab_b200 as ab

        names = ("table", "length", "k", "v", "ksum", "mass", "pos")
        t = {x: st[x] for x in names if x in st}
        t.setdefault("v", t["k"])  # scores and masses read no values
        st["cache"] = ab.KVCache(**t)
    return st["cache"]


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"append": _append, "score": _score, "attn": _attn, "mass": _mass, "evict": _evict}[op](st)
    import block_sparse_attention_ab_b200 as ab

    c = _cache(st)
    if op == "append":
        ab.cache_append(c, st["k_new"], st["v_new"], n_new=st["n"], sel=st["sel"], start=st["start"],
                        pos=st["pos0"])
        return [c.k, c.v, c.mass, c.pos, c.ksum, c.length]
    if op == "score":
        first, recent = _always(st["case"])
        return ab.cache_score(c, st["q"], n_tok=st["n"], per_token=st["case"]["per_token"],
                              first=first, recent=recent)
    if op == "attn":
        out, lse = ab.cache_attn(c, st["q"], st["k_new"], st["v_new"], n_tok=st["n"], tree=st.get("tree"),
                                 idx=st.get("idx"), cnt=st.get("cnt"), w=st.get("w"), want_lse=True)
        return [out, lse]
    if op == "mass":
        return ab.cache_mass(c, st["q"], st["lse"], n_tok=st["n"], out=st["out"])
    n = st["case"]["budget"]
    src, count = ab.cache_keep(c, n, recent=min(64, n // 2), next_pos=st["next_pos"], score=st["mass0"],
                               pos=st["pos0"], length=st["len0"])
    ab.cache_compact(c, src, count)
    return [src, count, c.k, c.v, c.mass, c.pos, c.ksum, c.length]


# --------------------------------------------------------------------------------------
# the operators' definitions in 64 bits, one sequence and head at a time
# --------------------------------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    B, Hq, Hk, d, T, page = (case[x] for x in ("B", "Hq", "Hk", "d", "T", "page"))
    op, G, f64 = case["op"], Hq // Hk, torch.float64
    L, n = _lengths(case), _counts(case)
    table = st["table"].long()

    def slots(x, b, h, count):
        """The first `count` slots of sequence b, head h."""
        p = table[b, : -(-count // page)]
        return x[p, h].reshape(p.numel() * page, *x.shape[3:])[:count]

    def summed(b, h, lp, count):
        """The key sums of pages lp of sequence b, of which `count` slots are valid."""
        rows = st["k"][table[b, lp], h].to(f64)
        there = lp.view(-1, 1) * page + torch.arange(page, device="cuda") < count
        return (rows * there.unsqueeze(-1)).sum(dim=1)

    if op == "append":
        ksum = st["ksum"].to(f64)
        for b in range(B):
            if n[b] == 0:
                continue
            at = L[b] + torch.arange(n[b], device="cuda")
            pg, off, sel = table[b, at // page], at % page, st["sel"][b, : n[b]].long()
            st["k"][pg, :, off] = st["k_new"][b][:, sel].transpose(0, 1)
            st["v"][pg, :, off] = st["v_new"][b][:, sel].transpose(0, 1)
            st["mass"][pg, :, off] = 0.0
            st["pos"][pg, :, off] = (st["pos0"][b] + torch.arange(n[b], device="cuda", dtype=torch.int32)).unsqueeze(1)
            lp = torch.arange(L[b] // page, (L[b] + n[b] - 1) // page + 1, device="cuda")
            for h in range(Hk):
                ksum[table[b, lp], h] = summed(b, h, lp, L[b] + n[b])
        return [st["k"], st["v"], st["mass"], st["pos"], ksum, st["len0"] + st["n"]]

    if op == "score":
        tp = T if case["per_token"] else 1
        res = torch.zeros(B, Hk, tp, table.shape[1], dtype=f64, device="cuda")
        for b in range(B):
            pages = -(-L[b] // page)
            if pages == 0 or n[b] == 0:
                continue
            size = torch.full((pages, 1), float(page), dtype=f64, device="cuda")
            size[-1] = L[b] - (pages - 1) * page
            for h in range(Hk):
                mean = st["ksum"][table[b, :pages], h].to(f64) / size
                for t in range(n[b]):
                    x = st["q"][b, h * G : (h + 1) * G, t].to(f64) @ mean.T / math.sqrt(d)
                    share = torch.softmax(x, dim=-1).mean(dim=0)
                    if tp > 1 or T == 1:
                        res[b, h, t, :pages] = share
                    else:
                        res[b, h, 0, :pages] += share / n[b]
            if case["weighted"]:
                live = n[b] if case["per_token"] else 1
                res[b, :, :live, :1] = 2.0
                res[b, :, :live, max(0, pages - 2) : pages] = 2.0
        return res

    if op == "attn":
        out = torch.zeros(B, Hq, T, d, dtype=f64, device="cuda")
        lse = torch.zeros(B, Hq, T, dtype=f64, device="cuda")
        for b in range(B):
            for h in range(Hk):
                k, v = (torch.cat([slots(st[x], b, h, L[b]), st[x + "_new"][b, h, : n[b]]]).to(f64) for x in "kv")
                s = st["q"][b, h * G : (h + 1) * G, : n[b]].to(f64) @ k.T / math.sqrt(d)
                shift = torch.zeros(n[b], k.shape[0], dtype=f64, device="cuda")
                if "idx" in st:
                    for t in range(st["idx"].shape[2] if st["idx"].shape[2] == 1 else n[b]):
                        row = torch.full((table.shape[1],), -math.inf, dtype=f64, device="cuda")
                        ids = st["idx"][b, h, t, : int(st["cnt"][b, h, t])].long()
                        row[ids] = torch.log(st["w"][b, h, t, : ids.numel()].to(f64)) if "w" in st else 0.0
                        each = row.repeat_interleave(page)[: L[b]]
                        if st["idx"].shape[2] == 1:
                            shift[:, : L[b]] = each
                        else:
                            shift[t, : L[b]] = each
                mine = st["tree"][b, : n[b], : n[b]] if "tree" in st else torch.ones(n[b], n[b], device="cuda").tril().bool()
                shift[:, L[b] :] = torch.where(mine, 0.0, -math.inf)
                s = s + shift
                lse[b, h * G : (h + 1) * G, : n[b]] = torch.logsumexp(s, dim=-1)
                out[b, h * G : (h + 1) * G, : n[b]] = torch.softmax(s, dim=-1) @ v
        return [out, lse]

    if op == "mass":
        res = st["out"].to(f64)
        for b in range(B):
            there = torch.arange(L[b], device="cuda")
            for h in range(Hk):
                s = st["q"][b, h * G : (h + 1) * G, : n[b]].to(f64) @ slots(st["k"], b, h, L[b]).to(f64).T / math.sqrt(d)
                p = torch.exp(s - st["lse"][b, h * G : (h + 1) * G, : n[b]].to(f64).unsqueeze(-1))
                last = L[b] - n[b] + torch.arange(n[b], device="cuda").view(-1, 1)
                got = torch.where(there <= last, p, 0.0).sum(dim=(0, 1)) + slots(st["mass"], b, h, L[b]).to(f64)
                res[table[b, there // page], h, there % page] = got
        return res

    keep_n = case["budget"]
    recent = min(64, keep_n // 2)
    src = torch.full((B, Hk, keep_n), -1, dtype=torch.int32, device="cuda")
    ksum = st["ksum"].to(f64)
    for b in range(B):
        m = min(L[b], keep_n)
        for h in range(Hk):
            x = slots(st["mass"], b, h, L[b]).clone()
            x[slots(st["pos"], b, h, L[b]) >= int(st["next_pos"][b]) - recent] = math.inf
            kept = torch.argsort(x, descending=True, stable=True)[:m].sort().values
            src[b, h, :m] = torch.arange(m, device="cuda", dtype=torch.int32)
            stay = torch.zeros(m, dtype=torch.bool, device="cuda")
            stay[kept[kept < m]] = True
            to, frm = torch.nonzero(~stay).flatten(), kept[kept >= m]
            src[b, h, to] = frm.int()
            a, z = (table[b, to // page], h, to % page), (table[b, frm // page], h, frm % page)
            for name in ("k", "v", "mass", "pos"):
                st[name][a] = st[name][z]
            dirty = to // page
            if m % page:
                dirty = torch.cat([dirty, dirty.new_tensor([m // page])])
            dirty = torch.unique(dirty)
            ksum[table[b, dirty], h] = summed(b, h, dirty, m)
    count = torch.tensor([min(x, keep_n) for x in L], dtype=torch.int32, device="cuda")
    return [src, count, st["k"], st["v"], st["mass"], st["pos"], ksum, count.clone()]
