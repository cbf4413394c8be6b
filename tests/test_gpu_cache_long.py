"""The tensor-core kernels of ab_cache_attn and ab_cache_mass over long caches: every CTA walks
tens of tiles, so that tile rings, buffers and barriers are used again and again, running
maxima rise along the walk, and a CTA goes from one head and sequence to the next. Against the
definitions of include/ab_attn.h in 64 bits, on the GPU.

Values that mark their place make a wrong tile show: v[s] is 1 in component (s / 64) mod d and 0
elsewhere, so an output component is the weight of every d-th unit of 64 slots, and its error is
relative to that weight: a probability rounded to the type (half a step), the logits' error and
the fp32 sums of the kernel, counted below. A unit that is taken twice, not at all or in
another's place is off by its whole weight."""

import math

import pytest
import torch

import block_sparse_attention_ab_b200 as ab
from cache_reference import F64, logit_error

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
SMS, UNIT = 148, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_attention_ab_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ab.lib()


class Long:
    """A cache on the GPU with shuffled pages. Keys grow by 2^(31/11) over every 32 units, from a
    unit to the one below it, which is the order the kernel walks in."""

    def __init__(self, lengths, Hk, d, page, dtype, seed):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.Hk, self.d, self.page, self.dtype = lengths, Hk, d, page, dtype
        self.B = len(lengths)
        self.max_pages = -(-max(lengths) // page) + 2
        need = [-(-n // page) for n in lengths]
        n_pages = sum(need) + 1
        order = torch.randperm(n_pages, generator=g, device="cuda")
        self.table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32, device="cuda")
        at = 0
        self.k = self.randn(n_pages, Hk, page, d)
        self.v = torch.zeros_like(self.k)
        for b, n in enumerate(need):
            pg = order[at : at + n]
            at += n
            self.table[b, :n] = pg.int()
            s = torch.arange(n * page, device="cuda")
            u = s // UNIT
            grow = 0.3 * 2.0 ** ((31 - u % 32).float() / 11)
            self.k[pg] = (self.k[pg].float() * grow.view(n, 1, page, 1)).to(dtype)
            mark = torch.zeros(n * page, d, dtype=dtype, device="cuda")
            mark[s, u % d] = 1
            self.v[pg] = mark.view(n, 1, page, d).expand(-1, Hk, -1, -1)
        self.length = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.mass = torch.zeros(n_pages, Hk, page, device="cuda")
        self.cache = ab.KVCache(k=self.k, v=self.v, table=self.table, length=self.length, mass=self.mass)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(self.dtype)

    def slots(self, t, b, h):
        n = self.lengths[b]
        x = t[self.table[b, : -(-n // self.page)].long(), h]
        return x.reshape(-1, *x.shape[2:])[:n]

    def tree(self, T):
        m = torch.zeros(self.B, T, T, dtype=torch.bool)
        g = torch.Generator().manual_seed(T)
        for b in range(self.B):
            for t in range(T):
                p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
                if p >= 0:
                    m[b, t] = m[b, p]
                m[b, t, t] = True
        return m.cuda()

    def plan(self, rows, share, weighted):
        idx = torch.full((self.B, self.Hk, rows, self.max_pages), -1, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(self.B, self.Hk, rows, dtype=torch.int32, device="cuda")
        w = torch.zeros(idx.shape, device="cuda")
        for b in range(self.B):
            pages = -(-self.lengths[b] // self.page)
            n = max(1, int(pages * share))
            pick = torch.rand(self.Hk, rows, pages, generator=self.g, device="cuda").argsort(-1)[..., :n]
            idx[b, :, :, :n] = pick.sort(-1).values.int()
            cnt[b] = n
            w[b, :, :, :n] = 1 + 19 * torch.rand(self.Hk, rows, n, generator=self.g, device="cuda")
        return idx, cnt, (w if weighted else None)

    def shift(self, plan, b, h, row):
        """ln of every slot's weight under a plan row, -inf outside it."""
        idx, cnt, w = plan
        n = int(cnt[b, h, row])
        of_page = torch.full((self.max_pages,), -math.inf, dtype=F64, device="cuda")
        of_page[idx[b, h, row, :n].long()] = 0.0 if w is None else w[b, h, row, :n].to(F64).log()
        return of_page[torch.arange(self.lengths[b], device="cuda") // self.page]


LENGTHS = [9000, 17001, 64, 20011, 5003, 12800]

ATTN = [
    # Hk, G, T, d, page, type: rows per key head G T
    (4, 3, 8, 128, 16, BF),     # 24: two sets of warps on the same rows
    (4, 4, 32, 64, 128, FP),    # 128
    (4, 8, 25, 128, 64, FP),    # 200: two halves
    (4, 4, 64, 64, 32, BF),     # 256
    (4, 5, 64, 128, 128, BF),   # 320: three halves, the last one half full
    (4, 3, 128, 64, 16, FP),    # 384
    (4, 7, 64, 128, 32, FP),    # 448: two tiles of two halves
]


@pytest.mark.parametrize("Hk,G,T,d,page,dtype", ATTN)
@pytest.mark.parametrize("use", ["all", "tree", "plan"])
def test_attn_many_tiles_a_cta(Hk, G, T, d, page, dtype, use):
    c = Long(LENGTHS, Hk, d, page, dtype, seed=T + d)
    n_tok = [max(1, T - 3 * b) for b in range(c.B)]
    _attn_case(c, G, T, n_tok, use)


@pytest.mark.parametrize("d,page,dtype", [(128, 64, BF), (64, 16, FP)])
def test_attn_many_tiles_plan_per_token(d, page, dtype):
    """Plan rows of 24 query heads each."""
    c = Long(LENGTHS, 4, d, page, dtype, seed=5)
    _attn_case(c, 24, 3, [3, 3, 2, 1, 3, 3], "plan_per_token")


def test_attn_tiles_whole_groups():
    """So many plan rows that every row is one CTA's, with the tensor-core kernel."""
    c = Long([900 + 7 * b for b in range(66)], 1, 64, 16, BF, seed=6)
    _attn_case(c, 24, 128, [128] * c.B, "plan_per_token", pick=[0, 31, 65])


def test_attn_more_row_tiles_than_sms():
    """200 tiles of 384 query rows, each one CTA's."""
    c = Long([700, 1300], 1, 64, 32, BF, seed=7)
    _attn_case(c, 600, 128, [128, 100], "all")


def _attn_case(c, G, T, n_tok, use, pick=None):
    q = c.randn(c.B, c.Hk * G, T, c.d, scale=1.5)
    k = c.randn(c.B, c.Hk, T, c.d, scale=0.3)
    v = torch.zeros_like(k)
    at = torch.arange(T, device="cuda")
    v[:, :, at, (c.d - 1 - at) % c.d] = 1
    tree = c.tree(T) if use == "tree" else None
    per_token = use == "plan_per_token"
    plan = c.plan(T if per_token else 1, 0.4, c.page != 32) if use.startswith("plan") else None
    idx, cnt, w = plan or (None, None, None)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = ab.cache_attn(c.cache, q, k, v, n_tok=torch.tensor(n_tok, dtype=torch.int32, device="cuda"), tree=tree,
                             idx=idx, cnt=cnt, w=w, want_lse=True, out_dtype=torch.float32, dev_flag=flag)
    assert ab.check_flag(flag) == 0
    u_p = torch.finfo(c.dtype).eps / 2
    # fp32 additions behind one another. A CTA's run: U units, of which a row's sum takes 12 each
    # (8 into one of four accumulators, 3 to join them) and an output 64, counted twice because
    # the tensor core may truncate; then the parts of at most SMS CTAs. Each rescaling of the sums
    # by a power is one more rounding and a base-2 exponential (2^-21): at most one per unit.
    units = sum(-(-n // UNIT) + -(-T // UNIT) for n in c.lengths) * c.Hk * (T if per_token else 1)
    ctas = max(1, SMS // -(-G * T // 128))  # of a row tile, at least
    U = -(-units // ctas) + 1 if not per_token else max(c.lengths) // UNIT + 2
    chain_l = (12 * U + SMS) * 2.0 ** -24 + U * 2.0 ** -21
    chain_o = (128 * U + SMS) * 2.0 ** -24 + U * 2.0 ** -21
    for b in pick if pick is not None else range(c.B):
        n = n_tok[b]
        assert bool((got[b, :, n:] == 0).all()) and bool((lse[b, :, n:] == 0).all())
        for h in range(c.Hk):
            keys, vals = c.slots(c.k, b, h), c.slots(c.v, b, h)
            allk = torch.cat([keys, k[b, h, :n]]).to(F64)
            allv = torch.cat([vals, v[b, h, :n]]).to(F64)
            for t0, t1 in ([(t, t + 1) for t in range(n)] if per_token else [(0, n)]):
                if per_token and pick is not None and t0 % 37:
                    continue
                rows = q[b, h * G : (h + 1) * G, t0:t1].reshape(-1, c.d).to(F64)  # (g, t)
                s = rows @ allk.T / math.sqrt(c.d)
                if plan is not None:
                    s[:, : c.lengths[b]] += c.shift(plan, b, h, t0 if per_token else 0)
                sees = tree[b, t0:t1, :n] if tree is not None else \
                    torch.arange(n, device="cuda") <= torch.arange(t0, t1, device="cuda").unsqueeze(1)
                s[:, c.lengths[b] :].masked_fill_(~sees.repeat(G, 1), -math.inf)
                ref_lse = torch.logsumexp(s, -1)
                p = torch.softmax(s, -1)
                ref = p @ allv
                e = logit_error(rows, allk) + 2.0 ** -22 * float(s[s > -math.inf].abs().max()) + 2.0 ** -21
                g_out = got[b, h * G : (h + 1) * G, t0:t1].reshape(-1, c.d).to(F64)
                g_lse = lse[b, h * G : (h + 1) * G, t0:t1].reshape(-1).to(F64)
                err = (g_lse - ref_lse).abs()
                lim = 2 * e + chain_l + 2.0 ** -21 + 2.0 ** -23 * ref_lse.abs()
                assert bool((err <= lim).all()), (b, h, float((err / lim).max()))
                # fp16 holds probabilities down to 2^-24 of what is 2^7 or more at the maximum
                tiny = allk.shape[0] * 2.0 ** -31 if c.dtype == FP else 0.0
                err = (g_out - ref).abs()
                lim = (u_p + 4 * e + 2 * chain_o) * ref + tiny + 1e-30
                assert bool((err <= lim).all()), (b, h, float((err / lim).max()))


MASS = [
    # Hk, G, T, d, page, type
    (4, 2, 32, 128, 16, BF),
    (4, 4, 50, 64, 128, FP),
    (4, 2, 100, 128, 64, FP),
    (4, 5, 100, 128, 32, BF),   # two passes of 256 rows
    (4, 8, 64, 64, 64, BF),
]


@pytest.mark.parametrize("Hk,G,T,d,page,dtype", MASS)
def test_mass_many_tiles_a_cta(Hk, G, T, d, page, dtype):
    c = Long(LENGTHS, Hk, d, page, dtype, seed=T + d)
    n_tok = [max(1, T - 3 * b) for b in range(c.B)]
    n_tok[2] = min(n_tok[2], c.lengths[2])
    q = c.randn(c.B, Hk * G, T, d, scale=1.5)
    lse = torch.zeros(c.B, Hk * G, T, device="cuda")
    refs = {}
    for b in range(c.B):
        n, L = n_tok[b], c.lengths[b]
        for h in range(Hk):
            keys = c.slots(c.k, b, h).to(F64)
            rows = q[b, h * G : (h + 1) * G, :n].reshape(-1, d).to(F64)
            s = rows @ keys.T / math.sqrt(d)
            sees = torch.arange(L, device="cuda") < L - n + 1 + torch.arange(n, device="cuda").unsqueeze(1)
            s.masked_fill_(~sees.repeat(G, 1), -math.inf)
            l32 = torch.logsumexp(s, -1).float()
            lse[b, h * G : (h + 1) * G, :n] = l32.view(G, n)
            p = torch.exp(s - l32.to(F64).unsqueeze(1)).sum(0)
            e = 2 * logit_error(rows, keys) + 2.0 ** -20 * (1 + float(s[s > -math.inf].abs().max())
                                                            + float(l32.abs().max()))
            refs[b, h] = p, p * (e + (n * G + 2) * 2.0 ** -24)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ab.cache_mass(c.cache, q, lse, n_tok=torch.tensor(n_tok, dtype=torch.int32, device="cuda"), dev_flag=flag)
    assert ab.check_flag(flag) == 0
    for (b, h), (p, tol) in refs.items():
        err = (c.slots(c.mass, b, h).to(F64) - p).abs()
        assert bool((err <= tol + 1e-30).all()), (b, h, float((err / (tol + 1e-30)).max()))
