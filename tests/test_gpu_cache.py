"""GPU tests of the key/value cache calls against their definitions in 64 bits
(tests/cache_reference.py): page sizes, head groups, types, strides, ragged batches, empty
sequences, trees, plans, rows that see nothing, and what must stay as it was.

Tolerances come from the arithmetic and are computed beside each reference value: fp32 sums
of exact 16-bit products, probabilities rounded once to the values' type before the second
product (half a step, finfo.eps / 2), the output rounded once more. Moves and selections are
exact."""

import math

import pytest
import torch

import block_sparse_attention_ab_b200 as ab
from cache_reference import F64, HostCache, attn, compact, keep, mass, score

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_attention_ab_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ab.lib()


def _flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _tree(B, T, g):
    """Random trees: each token's parent is an earlier token or the context."""
    m = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            if p >= 0:
                m[b, t] = m[b, p]
            m[b, t, t] = True
    return m


def _plan(c, rows, budget, weighted, g, empty=()):
    idx = torch.full((c.B, c.Hk, rows, c.max_pages), -1, dtype=torch.int32)
    cnt = torch.zeros(c.B, c.Hk, rows, dtype=torch.int32)
    w = torch.zeros(idx.shape)
    for b in range(c.B):
        pages = -(-int(c.length[b]) // c.page)
        for h in range(c.Hk):
            for t in range(rows):
                n = 0 if (b, h, t) in empty else min(budget, pages)
                cnt[b, h, t] = n
                idx[b, h, t, :n] = torch.randperm(pages, generator=g)[:n].sort().values.int()
                w[b, h, t, :n] = 1 + 19 * torch.rand(n, generator=g)
    return idx, cnt, (w if weighted else None)


def _check_attn(got, lse, ref, out_dtype):
    out, ref_lse, tol, tol_lse = ref
    got, lse = got.cpu().to(F64), lse.cpu().to(F64)
    u_out = torch.finfo(out_dtype).eps / 2
    err = (got - out).abs()
    lim = tol + u_out * (out.abs() + tol) + 1e-7
    assert bool((err <= lim).all()), float((err - lim).max())
    assert torch.equal(lse == -math.inf, ref_lse == -math.inf)
    fin = ref_lse > -math.inf
    e = (lse[fin] - ref_lse[fin]).abs()
    assert bool((e <= tol_lse[fin] + 2.0 ** -23 * ref_lse[fin].abs()).all()), float(e.max())


CASES = [
    # lengths, Hk, G, d, page, T, type
    ([1], 1, 1, 128, 16, 1, BF),
    ([0, 5, 64], 2, 3, 64, 16, 1, FP),
    ([200, 1, 0, 333], 2, 4, 128, 32, 1, BF),
    ([517, 128], 3, 8, 128, 64, 1, FP),
    ([129, 255], 1, 12, 64, 128, 1, BF),
    ([700], 2, 5, 128, 128, 7, BF),
    ([65, 0], 2, 2, 64, 64, 33, FP),
    ([300, 40], 1, 3, 128, 16, 64, BF),
    ([131], 2, 1, 128, 32, 128, FP),
    ([2100, 4095, 1], 2, 2, 64, 16, 2, BF),
    ([90, 600], 1, 20, 128, 64, 9, FP),
    ([257], 1, 2, 128, 128, 100, BF),
    # more than one half of 128 query rows, and rows in the last half for some sequences only
    ([300, 900, 64], 1, 3, 128, 64, 86, FP),
    ([1100, 33], 2, 5, 128, 32, 70, BF),
    ([500], 1, 4, 64, 16, 127, BF),
    ([1300, 2], 1, 12, 64, 128, 50, FP),
    ([200], 1, 32, 128, 64, 12, BF),
]


@pytest.mark.parametrize("lengths,Hk,G,d,page,T,dtype", CASES)
@pytest.mark.parametrize("use", ["all", "tree", "plan", "plan_per_token"])
def test_attn_against_definition(lengths, Hk, G, d, page, T, dtype, use):
    c = HostCache(lengths, Hk, d, page, dtype, seed=T + 7 * d + page)
    B = len(lengths)
    q = c.randn(B, Hk * G, T, d, scale=1.5)
    k, v = c.randn(B, Hk, T, d), c.randn(B, Hk, T, d)
    n_tok = torch.tensor([max(0, T - 2 * b) for b in range(B)], dtype=torch.int32)
    tree = _tree(B, T, c.g) if use != "all" else None
    plan, per_token = None, False
    if use.startswith("plan"):
        per_token = use == "plan_per_token"
        plan = _plan(c, T if per_token else 1, 3, page != 32, c.g, empty={(0, 0, 0)})
        per_token = plan[0].shape[2] == T  # one token: the two forms are one
    flag = _flag()
    idx, cnt, w = _gpu(*plan) if plan else (None, None, None)
    qg, kg, vg, ng = _gpu(q, k, v, n_tok)
    gc = c.to_gpu()
    got, lse = ab.cache_attn(gc, qg, kg, vg, n_tok=ng, tree=None if tree is None else tree.cuda(), idx=idx,
                             cnt=cnt, w=w, want_lse=True, dev_flag=flag)
    f32, lse2 = ab.cache_attn(gc, qg, kg, vg, n_tok=ng, tree=None if tree is None else tree.cuda(), idx=idx,
                              cnt=cnt, w=w, want_lse=True, out_dtype=torch.float32, dev_flag=flag)
    assert ab.check_flag(flag) == 0
    ref = attn(c, q, k, v, n_tok, tree, plan, per_token)
    _check_attn(got, lse, ref, dtype)
    _check_attn(f32, lse2, ref, torch.float32)
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", ["phd"])
def test_attn_strides(layout):
    """[n_pages, page, Hk, d] storage with padded rows; [B, T, H, d] tokens."""
    c = HostCache([77, 130], 3, 64, 16, BF, seed=3, layout=layout)
    q, k, v = c.randn(2, 5, 6, 64), c.randn(2, 5, 3, 64), c.randn(2, 5, 3, 64)
    q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    got, lse = ab.cache_attn(c.to_gpu(), *(t.cuda() for t in (q, k, v)), want_lse=True)
    _check_attn(got, lse, attn(c, q, k, v), BF)


def test_attn_rows_that_see_nothing_and_rows_behind():
    c = HostCache([40, 0], 2, 64, 16, BF, seed=4)
    q, k, v = c.randn(2, 4, 3, 64), c.randn(2, 2, 3, 64), c.randn(2, 2, 3, 64)
    tree = torch.zeros(2, 3, 3, dtype=torch.bool)
    tree[0, 1, 0] = True
    n_tok = torch.tensor([3, 2], dtype=torch.int32)
    out = torch.full((2, 4, 3, 64), 7.0, dtype=BF, device="cuda")
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), k.cuda(), v.cuda(), n_tok=n_tok.cuda(), tree=tree.cuda(),
                             want_lse=True, out=out)
    _check_attn(got, lse, attn(c, q, k, v, n_tok, tree), BF)
    assert bool((got[1] == 0).all()) and bool((lse[1, :, :2] == -math.inf).all()) and bool((lse[1, :, 2] == 0).all())
    # no new tokens at all: the context alone
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), want_lse=True)
    _check_attn(got, lse, attn(c, q), BF)


def test_attn_nothing_behind_a_sequence_is_read():
    """NaN in every row that no sequence owns and in tokens behind n_tok changes nothing."""
    c = HostCache([45, 100, 0], 2, 128, 32, FP, spare=3, seed=5)
    q, k, v = c.randn(3, 4, 5, 128), c.randn(3, 2, 5, 128), c.randn(3, 2, 5, 128)
    n_tok = torch.tensor([5, 2, 1], dtype=torch.int32)
    ref = attn(c, q, k, v, n_tok)
    owned = torch.zeros(c.n_pages, c.page, dtype=torch.bool)
    for b in range(3):
        s = torch.arange(int(c.length[b]))
        owned[c.table[b, s // c.page].long(), s % c.page] = True
    for t in (c.k, c.v):
        t.permute(0, 2, 1, 3)[~owned] = math.nan
    for b in range(3):
        for t in (k, v, q):
            t[b, :, int(n_tok[b]):] = math.nan
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), k.cuda(), v.cuda(), n_tok=n_tok.cuda(), want_lse=True)
    _check_attn(got, lse, ref, FP)


@pytest.mark.parametrize("scale", [30.0, 1e-3])
def test_attn_large_and_small_logits(scale):
    c = HostCache([500], 1, 128, 64, BF, seed=6, scale=scale)
    q, k, v = c.randn(1, 4, 2, 128), c.randn(1, 1, 2, 128, scale=scale), c.randn(1, 1, 2, 128)
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check_attn(got, lse, attn(c, q, k, v), BF)


def test_attn_long_uniform_tail_in_fp16():
    """One heavy key and 60000 keys e^-14 below it: their probabilities are small in fp16."""
    L = 60000
    c = HostCache([L], 1, 64, 128, FP, seed=7)
    c.k.zero_()
    q = torch.zeros(1, 1, 1, 64, dtype=FP)
    q[..., 0] = 8.0
    heavy = c.table[0, 100]
    c.k[heavy, 0, 5, 0] = 14.0  # logit 14
    c.v.copy_(c.v.abs())
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), want_lse=True, out_dtype=torch.float32)
    kf, vf = c.slots("k", 0, 0, L).to(F64), c.slots("v", 0, 0, L).to(F64)
    s = q[0, 0].to(F64) @ kf.T / 8.0
    ref = torch.softmax(s, -1) @ vf
    # every probability is off by half a step at most: 2^-11
    assert bool(((got.cpu().to(F64)[0, 0] - ref).abs() <= 2.0 ** -11 * ref + 2.0 ** -16).all())


def test_attn_bits_repeat_and_whole_groups_agree():
    c = HostCache([3000, 100, 2222], 2, 128, 64, BF, seed=8)
    q, k, v = (t.cuda() for t in (c.randn(3, 10, 2, 128), c.randn(3, 2, 2, 128), c.randn(3, 2, 2, 128)))
    g = c.to_gpu()
    a, la = ab.cache_attn(g, q, k, v, want_lse=True)
    for _ in range(3):
        b, lb = ab.cache_attn(g, q, k, v, want_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_attn_many_plan_rows():
    """More plan rows than the run-of-units form scans: every row whole in one CTA."""
    B, Hk, T = 9, 8, 128
    c = HostCache([70 + b for b in range(B)], Hk, 64, 16, BF, seed=9)
    q, k, v = c.randn(B, Hk, T, 64), c.randn(B, Hk, T, 64), c.randn(B, Hk, T, 64)
    plan = _plan(c, T, 2, True, c.g)
    assert B * Hk * T > 8192
    got, lse = ab.cache_attn(c.to_gpu(), q.cuda(), k.cuda(), v.cuda(), idx=plan[0].cuda(), cnt=plan[1].cuda(),
                             w=plan[2].cuda(), want_lse=True)
    pick = [0, 4, 8]
    sub = HostCache([70 + b for b in range(B)], Hk, 64, 16, BF, seed=9)
    sub.B = len(pick)
    sub.table, sub.length = c.table[pick], c.length[pick]
    ref = attn(sub, q[pick], k[pick], v[pick], None, None, tuple(t[pick] for t in plan), True)
    _check_attn(got[pick], lse[pick], ref, BF)


def test_attn_flags():
    c = HostCache([100], 1, 64, 32, BF, seed=10)
    q = c.randn(1, 2, 1, 64).cuda()
    base = c.to_gpu()

    def run(cache, **kw):
        flag = _flag()
        out = ab.cache_attn(cache, q, dev_flag=flag, **kw)
        return out, ab.check_flag(flag)

    clean, bits = run(base)
    assert bits == 0
    # a table entry outside the pool: its page is skipped
    bad = HostCache([100], 1, 64, 32, BF, seed=10)
    bad.table[0, 1] = c.n_pages
    assert run(bad.to_gpu())[1] == ab.FLAG_BAD_INDEX
    long = HostCache([100], 1, 64, 32, BF, seed=10)
    long.length[0] = 10 ** 6
    assert run(long.to_gpu())[1] & ab.FLAG_BAD_INDEX
    idx = torch.full((1, 1, 1, c.max_pages), -1, dtype=torch.int32)
    idx[0, 0, 0, :3] = torch.tensor([0, c.max_pages, 2])
    cnt = torch.tensor([[[3]]], dtype=torch.int32)
    got, bits = run(base, idx=idx.cuda(), cnt=cnt.cuda())
    assert bits == ab.FLAG_BAD_INDEX
    idx[0, 0, 0, :2] = torch.tensor([0, 2])
    two = run(base, idx=idx.cuda(), cnt=torch.tensor([[[2]]], dtype=torch.int32).cuda())
    assert two[1] == 0 and bool(((got - two[0]).abs() <= 2.0 ** -7 * two[0].abs()).all())
    w = torch.ones(1, 1, 1, c.max_pages)
    w[0, 0, 0, 1] = -1.0
    assert run(base, idx=idx.cuda(), cnt=torch.tensor([[[2]]], dtype=torch.int32).cuda(), w=w.cuda())[1] == \
        ab.FLAG_BAD_WEIGHT
    # pages of the plan behind the sequence take no part and raise nothing
    idx[0, 0, 0, :3] = torch.tensor([0, 2, c.max_pages - 1])
    got, bits = run(base, idx=idx.cuda(), cnt=cnt.cuda())
    assert bits == 0 and bool(((got - two[0]).abs() <= 2.0 ** -7 * two[0].abs()).all())


# ------------------------------------------------------------------------------- scores


@pytest.mark.parametrize("lengths,Hk,G,d,page,T,dtype", CASES)
@pytest.mark.parametrize("per_token", [True, False])
def test_score_against_definition(lengths, Hk, G, d, page, T, dtype, per_token):
    c = HostCache(lengths, Hk, d, page, dtype, seed=T + d)
    B = len(lengths)
    q = c.randn(B, Hk * G, T, d)
    n_tok = torch.tensor([max(0, T - 2 * b) for b in range(B)], dtype=torch.int32)
    flag = _flag()
    first, recent = (1, 2) if page != 32 else (0, 0)
    got = ab.cache_score(c.to_gpu(), q.cuda(), n_tok=n_tok.cuda(), per_token=per_token, first=first,
                         recent=recent, dev_flag=flag)
    assert ab.check_flag(flag) == 0
    ref, rel = score(c, q, n_tok, per_token, first, recent)
    assert bool(((got.cpu().to(F64) - ref).abs() <= rel * ref + 1e-30).all())
    # the rows go to the selections as they are
    idx, cnt, w = ab.select(got, 2, "topk", dev_flag=flag)
    ab.select(got, 2, "sip", dev_flag=flag)
    assert ab.check_flag(flag) == 0


def test_score_many_pages():
    """16-token pages of one long sequence: every CTA of the cluster holds many pages."""
    c = HostCache([16 * 40000 - 5], 1, 64, 16, BF, seed=1, max_pages=65536)
    q = c.randn(1, 3, 2, 64)
    ref, rel = score(c, q, None, True)
    got = ab.cache_score(c.to_gpu(), q.cuda()).cpu().to(F64)
    assert bool(((got - ref).abs() <= rel * ref + 1e-30).all())
    one, rel = score(c, q, None, False)
    got = ab.cache_score(c.to_gpu(), q.cuda(), per_token=False).cpu().to(F64)
    assert bool(((got - one).abs() <= rel * one + 1e-30).all())


# ------------------------------------------------------------------------------- append


@pytest.mark.parametrize("Hk,d,page,dtype", [(1, 64, 16, BF), (3, 128, 32, FP), (2, 64, 64, FP), (2, 128, 128, BF)])
def test_append_writes_and_sums(Hk, d, page, dtype):
    lengths = [0, 5, page - 1, 2 * page, 3 * page + 7]
    c = HostCache(lengths, Hk, d, page, dtype, spare=60, max_pages=12, seed=2, layout="phd")
    T = 2 * page + 3
    n = torch.tensor([T, 1, 2, 0, T - 4], dtype=torch.int32)
    for b in range(5):
        c.allocate(b, lengths[b] + T)
    k, v = c.randn(5, Hk, T, d), c.randn(5, Hk, T, d)
    sel = torch.stack([torch.randperm(T, generator=c.g) for _ in range(5)]).int()
    pos0 = torch.tensor([100, 200, 300, 400, 500], dtype=torch.int32)
    g = c.to_gpu()
    flag = _flag()
    before = {x: getattr(g, x).clone() for x in ("k", "v", "mass", "pos", "ksum")}
    ab.cache_append(g, k.cuda(), v.cuda(), n_new=n.cuda(), sel=sel.cuda(), pos=pos0.cuda(), dev_flag=flag)
    assert ab.check_flag(flag) == 0
    assert g.length.tolist() == [a + int(b) for a, b in zip(lengths, n)]
    for b in range(5):
        for i in range(int(n[b])):
            s = lengths[b] + i
            at = (int(c.table[b, s // page]), slice(None), s % page)
            for x, new in (("k", k), ("v", v)):
                before[x][at] = new[b, :, int(sel[b, i])].cuda()
            before["mass"][at] = 0
            before["pos"][at] = int(pos0[b]) + i
    for x in ("k", "v", "mass", "pos"):
        assert torch.equal(getattr(g, x), before[x]), x
    got = g.ksum.cpu().to(F64)
    for b in range(5):
        L = lengths[b] + int(n[b])
        for lp in range(c.max_pages):
            pg = int(c.table[b, lp])
            if pg < 0:
                continue
            if int(n[b]) and lengths[b] // page <= lp and lp * page < L:
                rows = g.k[pg, :, : min(page, L - lp * page)].cpu().to(F64)
                assert bool(((got[pg] - rows.sum(1)).abs() <= page * 2.0 ** -24 * rows.abs().sum(1)).all())
            else:
                assert torch.equal(g.ksum[pg], before["ksum"][pg])


def test_append_sums_do_not_depend_on_the_steps():
    """One call, token by token, and a rollback give the same bits."""
    def fresh():
        c = HostCache([0], 2, 128, 64, BF, spare=8, max_pages=4, seed=3)
        c.allocate(0, 200)
        return c, c.to_gpu()
    c, one = fresh()
    _, many = fresh()
    k, v = c.randn(1, 2, 200, 128).cuda(), c.randn(1, 2, 200, 128).cuda()
    ab.cache_append(one, k, v)
    for a, z in ((0, 1), (1, 2), (2, 70), (70, 71), (71, 199), (199, 200)):
        ab.cache_append(many, k[:, :, a:z], v[:, :, a:z])
    assert one.length.item() == many.length.item() == 200
    for x in ("k", "v", "ksum", "pos"):
        assert torch.equal(getattr(one, x), getattr(many, x)), x
    # drafted tokens taken back: the sums are those of the tokens that stay
    ab.cache_append(many, v[:, :, :90], k[:, :, :90], start=torch.tensor([110], dtype=torch.int32, device="cuda"))
    ab.cache_append(many, k[:, :, 110:], v[:, :, 110:], start=torch.tensor([110], dtype=torch.int32, device="cuda"))
    for x in ("k", "v", "ksum", "pos"):
        assert torch.equal(getattr(one, x), getattr(many, x)), x


def test_append_limits():
    c = HostCache([30, 3], 1, 64, 16, BF, spare=4, max_pages=2, seed=4)
    c.allocate(1, 32)
    g = c.to_gpu()
    k, v = c.randn(2, 1, 8, 64).cuda(), c.randn(2, 1, 8, 64).cuda()
    old = g.k.clone()
    flag = _flag()
    ab.cache_append(g, k, v, dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_CACHE_FULL
    assert g.length.tolist() == [32, 11]
    assert torch.equal(g.k[int(c.table[0, 1]), 0, 14:], k[0, 0, :2])
    flag.zero_()
    ab.cache_append(g, k, v, start=torch.tensor([-1, 33], dtype=torch.int32, device="cuda"), dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_BAD_INDEX and g.length.tolist() == [32, 11]
    flag.zero_()
    sel = torch.full((2, 8), 8, dtype=torch.int32, device="cuda")
    ab.cache_append(g, k, v, n_new=torch.tensor([0, 1], dtype=torch.int32, device="cuda"), sel=sel, dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_BAD_INDEX
    assert bool((g.k[int(c.table[1, 0]), 0, 11] == 0).all())
    flag.zero_()
    hole = HostCache([16], 1, 64, 16, BF, spare=4, max_pages=3, seed=4).to_gpu()  # no second page
    ab.cache_append(hole, k[:1], v[:1], dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_BAD_INDEX
    assert torch.equal(old[int(c.table[0, 0])], g.k[int(c.table[0, 0])])


# --------------------------------------------------------------------------------- mass


@pytest.mark.parametrize("lengths,Hk,G,d,page,T,dtype", [
    ([1], 1, 1, 128, 16, 1, BF),
    ([70, 5, 300], 2, 3, 64, 16, 4, FP),
    ([200, 0, 333], 2, 4, 128, 32, 1, BF),
    ([517, 128], 1, 8, 128, 64, 40, FP),
    ([129, 255], 1, 12, 64, 128, 3, BF),
    ([2100, 64], 1, 2, 64, 16, 2, BF),
    # more than 32 query rows, for some sequences only; more than one pass of 256
    ([500, 90, 128], 2, 3, 128, 16, 60, BF),
    ([1000, 3], 1, 12, 64, 32, 90, FP),
    ([129, 700], 2, 5, 128, 128, 70, FP),
    ([64, 0, 65], 3, 8, 64, 64, 33, BF),
])
@pytest.mark.parametrize("use", ["all", "plan", "plan_per_token"])
def test_mass_against_definition(lengths, Hk, G, d, page, T, dtype, use):
    c = HostCache(lengths, Hk, d, page, dtype, seed=T + page)
    B = len(lengths)
    q = c.randn(B, Hk * G, T, d)
    n_tok = torch.tensor([min(n, max(0, T - b)) for b, n in enumerate(lengths)], dtype=torch.int32)
    sel = torch.stack([torch.randperm(T, generator=c.g) for _ in range(B)]).int()
    lse = 3 + torch.rand(B, Hk * G, T, generator=c.g)
    lse[0, 0, 0] = -math.inf
    plan, per_token = None, False
    if use != "all":
        per_token = use == "plan_per_token"
        plan = _plan(c, T if per_token else 1, 3, page != 32, c.g)
        per_token = plan[0].shape[2] == T
    idx, cnt, w = _gpu(*plan) if plan else (None, None, None)
    g = c.to_gpu()
    flag = _flag()
    out = torch.full_like(g.mass, 123.0)
    old = g.mass.clone()
    ab.cache_mass(g, q.cuda(), lse.cuda(), n_tok=n_tok.cuda(), sel=sel.cuda(), idx=idx, cnt=cnt, w=w, out=out,
                  dev_flag=flag)
    assert ab.check_flag(flag) == 0 and torch.equal(g.mass, old)
    ref, tol = mass(c, q, lse, n_tok, sel, plan, per_token)
    owned = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b in range(B):
        s = torch.arange(lengths[b])
        owned[c.table[b, s // page].long(), s % page] = True
    owned = owned.unsqueeze(1).expand(-1, Hk, -1)
    got = out.cpu().to(F64)
    assert bool((got[~owned] == 123.0).all())
    assert bool(((got - ref).abs() <= tol + 1e-7)[owned].all())
    # in place: the same values, the rest untouched
    ab.cache_mass(g, q.cuda(), lse.cuda(), n_tok=n_tok.cuda(), sel=sel.cuda(), idx=idx, cnt=cnt, w=w)
    assert torch.equal(g.mass.cpu()[owned], out.cpu()[owned])
    assert torch.equal(g.mass.cpu()[~owned], old.cpu()[~owned])


def test_mass_many_rows_adds_up():
    """More query rows than one pass holds; a row's weights over all slots sum to 1."""
    c = HostCache([400], 1, 64, 64, BF, seed=11)
    T, G = 100, 5
    q = c.randn(1, G, T, 64)
    g = c.to_gpu()
    keys = c.slots("k", 0, 0, 400).to(F64)
    s = q[0].to(F64) @ keys.T / 8.0
    sees = torch.arange(400) < 300 + torch.arange(T).unsqueeze(1) + 1
    lse = torch.logsumexp(s.masked_fill(~sees, -math.inf), -1).float().unsqueeze(0)
    out = torch.zeros_like(g.mass)
    g.mass.zero_()
    ab.cache_mass(g, q.cuda(), lse.cuda(), out=out)
    ref, tol = mass(c, q, lse)
    ref = ref - c.mass.to(F64)
    got = out.cpu().to(F64)
    assert bool(((got - ref).abs() <= tol + 1e-7).all())
    assert abs(float(got.sum()) - T * G) <= 1e-4 * T * G


# ------------------------------------------------------------------------------ eviction


@pytest.mark.parametrize("lengths,Hk,page,budget,recent", [
    ([1], 1, 16, 1, 0),
    ([5, 0, 40], 2, 16, 7, 2),
    ([300, 64, 65], 2, 32, 64, 0),
    ([1000, 999], 3, 64, 257, 40),
    ([5000, 4097, 4096], 1, 128, 4096, 100),
    ([40000], 1, 16, 12345, 1000),
    ([400000, 30], 1, 16, 200001, 1000),  # more than a cluster of CTAs holds
])
@pytest.mark.parametrize("ties", [False, True])
def test_keep_and_compact(lengths, Hk, page, budget, recent, ties):
    c = HostCache(lengths, Hk, 64, page, BF, seed=budget)
    if ties:  # few distinct values, zeros and infinities among them
        c.mass = torch.tensor([0.0, -0.0, 1.5, 1e-42, 3e38, math.inf])[
            torch.randint(0, 6, c.mass.shape, generator=c.g)]
    next_pos = torch.tensor([2 * n + 3 for n in lengths], dtype=torch.int32)
    for b, n in enumerate(lengths):
        for h in range(Hk):
            p = torch.randperm(2 * n + 3, generator=c.g)[:n].int()
            s = torch.arange(n)
            c.pos[c.table[b, s // page].long(), h, s % page] = p
    g = c.to_gpu()
    flag = _flag()
    src, count = ab.cache_keep(g, budget, recent=recent, next_pos=next_pos.cuda(), dev_flag=flag)
    ref_src, ref_count = keep(c, budget, recent, next_pos)
    assert torch.equal(count.cpu(), ref_count)
    assert torch.equal(src.cpu(), ref_src)
    old_sum = g.ksum.clone()
    ab.cache_compact(g, src, count, dev_flag=flag)
    assert ab.check_flag(flag) == 0
    due = compact(c, ref_src, ref_count)
    for x in ("k", "v", "mass", "pos", "length"):
        assert torch.equal(getattr(g, x).cpu(), getattr(c, x)), x
    touched = torch.zeros(c.n_pages, Hk, dtype=torch.bool)
    for pg, h, rows in due:
        touched[pg, h] = True
        x = c.k[pg, h, :rows].to(F64)
        got = g.ksum[pg, h].cpu().to(F64)
        assert bool(((got - x.sum(0)).abs() <= page * 2.0 ** -24 * x.abs().sum(0)).all())
    assert torch.equal(g.ksum.cpu()[~touched], old_sum.cpu()[~touched])
    # a second pass on the compacted cache moves nothing
    src, count = ab.cache_keep(g, budget)
    assert torch.equal(src.cpu().clamp(min=0),
                       torch.where(torch.arange(budget) < ref_count.view(-1, 1, 1), torch.arange(budget), 0)
                       .expand_as(ref_src).int())


def test_keep_flags_and_bad_moves():
    c = HostCache([50], 1, 64, 16, BF, seed=1)
    c.mass[int(c.table[0, 1]), 0, 3] = -1.0
    c.mass[int(c.table[0, 2]), 0, 0] = math.nan
    g = c.to_gpu()
    flag = _flag()
    src, count = ab.cache_keep(g, 20, dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_BAD_SCORE
    c.mass = torch.where(c.mass >= 0, c.mass, 0.0)
    assert torch.equal(src.cpu(), keep(c, 20)[0])
    k = g.k.clone()
    flag.zero_()
    bad = torch.arange(20, dtype=torch.int32).view(1, 1, 20).clone()
    bad[0, 0, 3], bad[0, 0, 4], bad[0, 0, 5] = 7, 10 ** 6, -1  # a slot that stays, and two that are none
    ab.cache_compact(g, bad.cuda(), torch.tensor([20], dtype=torch.int32, device="cuda"), dev_flag=flag)
    assert ab.check_flag(flag) == ab.FLAG_BAD_INDEX
    assert torch.equal(g.k, k) and g.length.item() == 20


# -------------------------------------------------------------------------- used together


def test_generation_with_selection_and_eviction():
    """The calls as a serving loop makes them, against a plain loop that keeps its own cache:
    scores, plan, attention, append of an accepted path, masses and eviction, 12 steps."""
    B, Hk, G, d, page, slots, T = 2, 2, 3, 64, 16, 96, 4
    c = HostCache([60, 23], Hk, d, page, BF, spare=24, max_pages=8, seed=21)
    for b in range(B):
        c.allocate(b, 128)
        for h in range(Hk):
            s = torch.arange(int(c.length[b]))
            c.pos[c.table[b, s // page].long(), h, s % page] = s.int()
    c.mass.zero_()
    g = c.to_gpu()
    # the sums of the tokens that are there: append nothing, page by page
    for b in range(B):
        for lp in range(-(-int(c.length[b]) // page)):
            rows = c.slots("k", b, 0, int(c.length[b]))
            for h in range(Hk):
                x = c.slots("k", b, h, int(c.length[b]))[lp * page : (lp + 1) * page].float().sum(0)
                c.ksum[int(c.table[b, lp]), h] = x
    g.ksum.copy_(c.ksum)
    next_pos = c.length.clone()
    flag = _flag()
    for step in range(12):
        q, k, v = c.randn(B, Hk * G, T, d), c.randn(B, Hk, T, d), c.randn(B, Hk, T, d)
        tree = _tree(B, T, c.g)
        qg, kg, vg, tg = _gpu(q, k, v, tree)
        per_token = step % 2 == 0
        sc = ab.cache_score(g, qg, per_token=per_token, first=1, recent=1, dev_flag=flag)
        ref, rel = score(c, q, None, per_token, 1, 1)
        assert bool(((sc.cpu().to(F64) - ref).abs() <= (rel + 1e-5) * ref + 1e-30).all())
        idx, cnt, w = ab.select(sc, 3, "sip", seed=step, dev_flag=flag)
        out, lse = ab.cache_attn(g, qg, kg, vg, tree=tg, idx=idx, cnt=cnt, w=w, want_lse=True, dev_flag=flag)
        plan = (idx.cpu(), cnt.cpu(), w.cpu())
        _check_attn(out, lse, attn(c, q, k, v, None, tree, plan, per_token), BF)
        # the accepted path: the last token's ancestors and itself
        n = tree[:, -1].sum(-1).int()
        sel = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            sel[b, : int(n[b])] = torch.nonzero(tree[b, -1]).flatten().int()
        ab.cache_append(g, kg, vg, n_new=n.cuda(), sel=sel.cuda(), pos=next_pos.cuda(), dev_flag=flag)
        for b in range(B):
            for i in range(int(n[b])):
                s = int(c.length[b]) + i
                at = (int(c.table[b, s // page]), slice(None), s % page)
                c.k[at], c.v[at] = k[b, :, int(sel[b, i])], v[b, :, int(sel[b, i])]
                c.mass[at], c.pos[at] = 0.0, int(next_pos[b]) + i
        c.length += n
        next_pos += n
        ab.cache_mass(g, qg, lse, n_tok=n.cuda(), sel=sel.cuda(), idx=idx, cnt=cnt, w=w, dev_flag=flag)
        ref, tol = mass(c, q, lse.cpu(), n, sel, plan, per_token)
        assert bool(((g.mass.cpu().to(F64) - ref).abs() <= tol + 1e-6).all())
        c.mass = g.mass.cpu()
        src, count = ab.cache_keep(g, slots, recent=8, next_pos=next_pos.cuda(), dev_flag=flag)
        rs, rc = keep(c, slots, 8, next_pos)
        assert torch.equal(src.cpu(), rs) and torch.equal(count.cpu(), rc)
        ab.cache_compact(g, src, count, dev_flag=flag)
        compact(c, rs, rc)
        for x in ("k", "v", "mass", "pos", "length"):
            assert torch.equal(getattr(g, x).cpu(), getattr(c, x)), x
        c.ksum = g.ksum.cpu()
        for b in range(B):  # every valid page's sum is that of its valid keys
            L = int(c.length[b])
            for lp in range(-(-L // page)):
                for h in range(Hk):
                    x = c.slots("k", b, h, L)[lp * page : (lp + 1) * page].to(F64)
                    got = c.ksum[int(c.table[b, lp]), h].to(F64)
                    assert bool(((got - x.sum(0)).abs() <= page * 2.0 ** -24 * x.abs().sum(0)).all())
    assert ab.check_flag(flag) == 0


def test_step_captured_and_replayed():
    """One token's step in a CUDA graph, on a side stream, replayed on changing inputs."""
    B, Hk, G, d, page = 2, 2, 2, 128, 32

    def fresh():
        c = HostCache([37, 5], Hk, d, page, BF, spare=12, max_pages=6, seed=31)
        for b in range(B):
            c.allocate(b, 192)
        return c, c.to_gpu()
    c, a = fresh()
    _, e = fresh()
    toks = [[c.randn(B, h, 1, d).cuda() for h in (Hk * G, Hk, Hk)] for _ in range(6)]
    q, k, v = (torch.zeros_like(t) for t in toks[0])
    side = torch.cuda.Stream()

    def step(cache, q, k, v):
        sc = ab.cache_score(cache, q, first=1)
        idx, cnt, w = ab.select(sc, 2, "topk")
        out, lse = ab.cache_attn(cache, q, k, v, idx=idx, cnt=cnt, want_lse=True)
        ab.cache_append(cache, k, v)
        ab.cache_mass(cache, q, lse, idx=idx, cnt=cnt)
        return out

    with torch.cuda.stream(side):
        step(fresh()[1], q, k, v)  # the library and the allocator warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(a, q, k, v)
    torch.cuda.synchronize()
    for t in toks:
        for dst, x in zip((q, k, v), t):
            dst.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(e, *t))
    for x in ("k", "v", "ksum", "mass", "length"):
        assert torch.equal(getattr(a, x), getattr(e, x)), x


def test_long_cache_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements per tensor: its last pages."""
    page, Hk, d = 128, 8, 128
    n_pages = 17000  # 2.2e9 elements, 4.5 GB each for keys and values
    k = torch.zeros(n_pages, Hk, page, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    use = [n_pages - 1, 0, n_pages - 2, 16400]
    c = HostCache([4 * page - 9], Hk, d, page, BF, seed=41)
    gk = c.k[c.table[0, :4].long()]
    gv = c.v[c.table[0, :4].long()]
    k[use], v[use] = gk.cuda(), gv.cuda()
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    ksum = torch.zeros(n_pages, Hk, d, device="cuda")
    mass_ = torch.zeros(n_pages, Hk, page, device="cuda")
    pos_ = torch.zeros(n_pages, Hk, page, dtype=torch.int32, device="cuda")
    g = ab.KVCache(k=k, v=v, table=table, length=c.length.cuda(), ksum=ksum, mass=mass_, pos=pos_)
    q, kn, vn = c.randn(1, 16, 2, d), c.randn(1, Hk, 2, d), c.randn(1, Hk, 2, d)
    out, lse = ab.cache_attn(g, q.cuda(), kn.cuda(), vn.cuda(), want_lse=True)
    _check_attn(out, lse, attn(c, q, kn, vn), BF)
    ab.cache_append(g, kn.cuda(), vn.cuda())
    assert torch.equal(k[16400, :, 119:121].cpu(), kn[0])
    ab.cache_mass(g, q.cuda(), lse)
    per_head = torch.stack([mass_[use, h].sum() for h in range(Hk)]).cpu()
    assert bool(((per_head - 4.0).abs() <= 1e-4).all())  # two tokens, two query heads each


# ---------------------------------------------------------------- other calls, other places


@pytest.mark.parametrize("T", [1, 30])
def test_attn_and_mass_on_expanded_heads(T):
    """One stored key head seen as three (stride 0): no tensor map, many rows or few."""
    c = HostCache([333, 50], 1, 128, 64, BF, seed=51)
    g = c.to_gpu()
    q, k, v = c.randn(2, 6, T, 128), c.randn(2, 3, T, 128), c.randn(2, 3, T, 128)
    wide = ab.KVCache(k=g.k.expand(-1, 3, -1, -1), v=g.v.expand(-1, 3, -1, -1), table=g.table, length=g.length,
                      mass=torch.zeros(c.n_pages, 3, 64, device="cuda"))
    c.Hk, c.k, c.v = 3, c.k.expand(-1, 3, -1, -1), c.v.expand(-1, 3, -1, -1)
    c.mass = torch.zeros(c.n_pages, 3, 64)
    out, lse = ab.cache_attn(wide, q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check_attn(out, lse, attn(c, q, k, v), BF)
    ab.cache_mass(wide, q.cuda(), lse)
    ref, tol = mass(c, q, lse.cpu())
    assert bool(((wide.mass.cpu().to(F64) - ref).abs() <= tol + 1e-7).all())
    for call in (lambda: ab.cache_append(wide, k.cuda(), v.cuda()),
                 lambda: ab.cache_compact(wide, *ab.cache_keep(wide, 8))):
        with pytest.raises(ab.AbError, match="UNSUPPORTED"):
            call()


def test_binding_refusals():
    c = HostCache([40, 20], 2, 64, 16, BF, spare=4, seed=52)
    g = c.to_gpu()
    q, k = c.randn(2, 4, 3, 64).cuda(), c.randn(2, 2, 3, 64).cuda()
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="q must be"):
        ab.cache_attn(g, q.half())
    with pytest.raises(ValueError, match="k must be"):
        ab.cache_attn(g, q, q, q)
    with pytest.raises(ValueError, match="k and v go together"):
        ab.cache_attn(g, q, k)
    with pytest.raises(ValueError, match="same number of tokens"):
        ab.cache_attn(g, q, k[:, :, :2], k[:, :, :2])
    with pytest.raises(TypeError, match="n_tok must be"):
        ab.cache_attn(g, q, n_tok=n.long())
    with pytest.raises(ValueError, match="n_tok must be on"):
        ab.cache_attn(g, q, n_tok=n.cpu())
    with pytest.raises(ValueError, match="tree must be"):
        ab.cache_attn(g, q, k, k, tree=torch.ones(2, 3, 4, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="idx needs cnt"):
        ab.cache_attn(g, q, idx=torch.zeros(2, 2, 1, c.max_pages, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="out_dtype"):
        ab.cache_attn(g, q, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        ab.cache_append(g, k.transpose(2, 3).contiguous().transpose(2, 3), k)
    with pytest.raises(ab.AbError, match="AB_ERR_SHAPE"):
        ab.cache_score(g, torch.zeros(2, 3, 1, 64, dtype=BF, device="cuda"))
    with pytest.raises(ab.AbError, match="AB_ERR_ALIGN"):
        ab.cache_attn(g, torch.zeros(2, 4, 3, 72, dtype=BF, device="cuda")[..., 4:68])
    with pytest.raises(ab.AbError, match="AB_ERR_WORKSPACE"):
        ab.cache_attn(g, q, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ab.AbError, match="AB_ERR_UNSUPPORTED"):
        ab.cache_append(g, k, k, start=g.length)
    with pytest.raises(ValueError, match="mass"):
        ab.cache_mass(ab.KVCache(k=g.k, v=g.v, table=g.table, length=g.length), q, torch.zeros(2, 4, 3, device="cuda"))
    with pytest.raises(ValueError, match="mass must be"):
        ab.KVCache(k=g.k, v=g.v, table=g.table, length=g.length, mass=g.mass[:, :1])
    with pytest.raises(ValueError, match="one shape"):
        ab.KVCache(k=g.k, v=g.v[:1], table=g.table, length=g.length)


@pytest.mark.parametrize("T", [1, 24])
def test_calls_on_two_streams_at_once(T):
    """Calls in flight on two streams, each with its own workspace, give what they give alone."""
    made = []
    for seed in (61, 62):
        c = HostCache([3000, 1999, 17], 2, 128, 64, BF, seed=seed)
        made.append((c.to_gpu(), *(x.cuda() for x in (c.randn(3, 10, T, 128), c.randn(3, 2, T, 128),
                                                      c.randn(3, 2, T, 128)))))
    alone = [ab.cache_attn(g, q, k, v, want_lse=True) for g, q, k, v in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ab.cache_attn(*made[i], want_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(l, alone[i][1])


def test_tree_step_captured_and_replayed():
    """A drafted tree's step (the tile kernels) in a graph, replayed on changing inputs."""
    B, Hk, G, d, page, T = 2, 2, 4, 64, 64, 16

    def fresh():
        c = HostCache([300, 65], Hk, d, page, FP, spare=12, max_pages=9, seed=71)
        for b in range(B):
            c.allocate(b, 570)
        return c, c.to_gpu()
    c, a = fresh()
    _, e = fresh()
    toks = [[c.randn(B, h, T, d).cuda() for h in (Hk * G, Hk, Hk)] + [_tree(B, T, c.g).cuda()] for _ in range(3)]
    q, k, v, tree = (torch.zeros_like(t) for t in toks[0])

    def step(cache, q, k, v, tree):
        out, lse = ab.cache_attn(cache, q, k, v, tree=tree, want_lse=True)
        ab.cache_append(cache, k, v)
        ab.cache_mass(cache, q, lse)
        return out

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(fresh()[1], q, k, v, tree)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(a, q, k, v, tree)
    torch.cuda.synchronize()
    for t in toks:
        for dst, x in zip((q, k, v, tree), t):
            dst.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(e, *t))
    for x in ("k", "v", "ksum", "mass", "length"):
        assert torch.equal(getattr(a, x), getattr(e, x)), x


def test_one_token_of_a_full_table_and_of_many_sequences():
    """Every slot of the table in use; 300 sequences of a few tokens, some empty."""
    c = HostCache([64, 63], 1, 64, 16, BF, max_pages=4, seed=81)
    q, k, v = c.randn(2, 2, 1, 64), c.randn(2, 1, 1, 64), c.randn(2, 1, 1, 64)
    out, lse = ab.cache_attn(c.to_gpu(), q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check_attn(out, lse, attn(c, q, k, v), BF)
    many = HostCache([(7 * b) % 40 for b in range(300)], 1, 64, 16, FP, seed=82)
    q, k, v = many.randn(300, 3, 1, 64), many.randn(300, 1, 1, 64), many.randn(300, 1, 1, 64)
    g = many.to_gpu()
    out, lse = ab.cache_attn(g, q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check_attn(out, lse, attn(many, q, k, v), FP)
    flag = _flag()
    sc = ab.cache_score(g, q.cuda(), dev_flag=flag)
    ref, rel = score(many, q)
    assert ab.check_flag(flag) == 0
    assert bool(((sc.cpu().to(F64) - ref).abs() <= rel * ref + 1e-30).all())


def test_captured_behind_copies_and_a_second_stream():
    """The calls' launches overlap the kernel before them; in a graph that may be a copy, a
    fill, or the join of two streams."""
    c = HostCache([200, 31], 2, 64, 32, BF, spare=12, max_pages=9, seed=91)
    for b in range(2):
        c.allocate(b, 288)
    g = c.to_gpu()
    src = [x.cuda() for x in (c.randn(2, 4, 2, 64), c.randn(2, 2, 2, 64), c.randn(2, 2, 2, 64))]
    q, k, v = (torch.empty_like(t) for t in src)
    start = g.length.clone()
    mass_out = torch.empty_like(g.mass)

    def step():
        q.copy_(src[0])  # a memory copy
        cur, other = torch.cuda.current_stream(), torch.cuda.Stream()
        other.wait_stream(cur)
        with torch.cuda.stream(other):
            k.copy_(src[1])
            v.copy_(src[2])
            mass_out.zero_()
        cur.wait_stream(other)
        out, lse = ab.cache_attn(g, q, k, v, want_lse=True)
        other.wait_stream(cur)
        with torch.cuda.stream(other):
            ab.cache_append(g, k, v, start=start)
            ab.cache_mass(g, q, lse, out=mass_out)
        cur.wait_stream(other)
        return out, lse

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ref = [t.clone() for t in step()] + [mass_out.clone()]
        g.length.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = step()
    for _ in range(3):
        for t in (q, k, v, out, lse, mass_out):
            t.fill_(7)
        g.length.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, lse, mass_out), ref):
            assert torch.equal(a, b)
        assert torch.equal(g.length, start + 2)
