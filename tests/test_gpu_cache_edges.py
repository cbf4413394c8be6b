"""GPU tests of the key/value cache calls at the edges of what their documentation allows:
capacities whose keys nearly fill the default shared memory, rollbacks that add nothing, counts
and indexes out of range, infinities and NaN where nothing looks, and handles whose tensors moved."""

import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import block_sparse_attention_ab_b200 as ab
from cache_reference import F64, HostCache, attn, mass

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_attention_ab_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ab.lib()


def _flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


_KEEP_ALONE = """
import sys
import torch
import block_sparse_attention_ab_b200 as ab
from cache_reference import HostCache, keep
Hk, slots = int(sys.argv[1]), int(sys.argv[2])
c = HostCache([slots], Hk, 64, 16, torch.bfloat16, seed=1, max_pages=slots // 16)
src, n = ab.cache_keep(c.to_gpu(), slots // 3)
ref, m = keep(c, slots // 3)
assert torch.equal(src.cpu(), ref) and torch.equal(n.cpu(), m)
print("kept")
"""


@pytest.mark.parametrize("Hk,slots", [(1, 45056), (40, 22528), (80, 11264)])
def test_keep_alone_in_a_process(Hk, slots):
    """Keys that fit the default limit of shared memory, but not beside the kernel's own arrays:
    no larger call has raised the limit before."""
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(HERE), HERE]))
    out = subprocess.run([sys.executable, "-c", _KEEP_ALONE, str(Hk), str(slots)], env=env, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0 and "kept" in out.stdout, out.stderr[-2000:]


def test_keep_of_two_sizes_from_two_threads():
    """Calls that need different amounts of shared memory, made by two host threads at once."""
    from block_sparse_attention_ab_b200.cache import AB_BF16, CacheStruct
    L = ab.lib()
    made = []
    for slots in (29696, 15360):  # 119 and 60 KB of keys
        pages = slots // 128
        held = torch.rand(pages, 148, 128, device="cuda"), torch.arange(pages, device="cuda").int(), _i32(slots)
        src, n, ws = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (14800, 1, 14800))
        s = CacheStruct(None, None, None, held[0].data_ptr(), None, held[1].data_ptr(), held[2].data_ptr(), 0, 0, 0, 0,
                        0, 0, 1, 148, 64, 128, pages, pages, AB_BF16)
        made.append((s, src, n, ws, torch.cuda.Stream(), held))
    torch.cuda.synchronize()
    codes = [set(), set()]

    def calls(i):
        s, src, n, ws, stream, _ = made[i]
        for _ in range(1500):
            codes[i].add(L.ab_cache_keep(s, 100, 0, None, None, None, None, src.data_ptr(), n.data_ptr(),
                                         ws.data_ptr(), ws.numel() * 4, None, stream.cuda_stream))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]


@pytest.mark.parametrize("page,d,dtype", [(16, 64, FP), (128, 128, BF)])
def test_rollback_that_adds_nothing(page, d, dtype):
    """Every drafted token of a sequence taken back: sums and scores are those of a cache that
    never held them."""
    def fresh():
        c = HostCache([0, 0, 0], 2, d, page, dtype, spare=12, max_pages=4, seed=3)
        for b in range(3):
            c.allocate(b, 4 * page)
        return c, c.to_gpu()
    c, a = fresh()
    _, e = fresh()
    k, v = c.randn(3, 2, 3 * page, d).cuda(), c.randn(3, 2, 3 * page, d).cuda()
    at = [page + 5, 2 * page, 2 * page + 1]  # in a page, at a page's end, one slot into a page
    ab.cache_append(a, k, v)
    flag, held = _flag(), (a.k.clone(), a.v.clone())
    ab.cache_append(a, v, k, n_new=_i32(0, 0, 0), start=_i32(*at), dev_flag=flag)
    ab.cache_append(e, k, v, n_new=_i32(*at))
    assert ab.check_flag(flag) == 0 and a.length.tolist() == e.length.tolist() == at
    for b in range(3):
        pages = c.table[b, : -(-at[b] // page)].long().cuda()
        assert torch.equal(a.ksum[pages], e.ksum[pages])
    assert torch.equal(a.k, held[0]) and torch.equal(a.v, held[1])
    q = c.randn(3, 4, 1, d).cuda()
    assert torch.equal(ab.cache_score(a, q), ab.cache_score(e, q))


def test_append_with_the_length_array():
    """length as start, position or count beside start is refused: the call writes it. Copies of
    it, and length as the count without start, do what they say."""
    c = HostCache([70, 33, 5], 4, 64, 16, BF, spare=30, seed=20, max_pages=10)
    for b in range(3):
        c.allocate(b, 160)
    g = c.to_gpu()
    k, v = c.randn(3, 4, 70, 64).cuda(), c.randn(3, 4, 70, 64).cuda()
    old = g.length.clone()
    for bad in (dict(start=g.length), dict(start=old, pos=g.length), dict(start=old, n_new=g.length)):
        with pytest.raises(ab.AbError, match="UNSUPPORTED"):
            ab.cache_append(g, k, v, **bad)
    assert torch.equal(g.length, old)
    ab.cache_append(g, k[:, :, :40], v[:, :, :40], start=old, pos=old.clone())
    assert torch.equal(g.length, old + 40)
    for b in range(3):
        s = torch.arange(int(old[b]), int(old[b]) + 40)
        pg = c.table[b, s // 16].long().cuda()
        assert torch.equal(g.pos[pg, :, (s % 16).cuda()].cpu(), s.int().unsqueeze(1).expand(-1, 4))
    g.length.copy_(old)
    ab.cache_append(g, k, v, n_new=g.length)
    assert torch.equal(g.length, 2 * old)


def test_keep_refuses_sizes_outside_32_bits():
    g = HostCache([40], 1, 64, 16, BF, seed=17).to_gpu()
    for budget in (0, -1, 5 - 2 ** 32, -2 ** 31 - 1, 2 ** 32 + 5, 2 ** 62):
        with pytest.raises((ValueError, ab.AbError)):
            ab.cache_keep(g, budget)
    for recent in (-1, 5 - 2 ** 32, 2 ** 32 + 5):
        with pytest.raises((ValueError, ab.AbError)):
            ab.cache_keep(g, 8, recent=recent, next_pos=_i32(40))


def test_sizes_past_32_bits_are_refused():
    c = HostCache([40], 1, 64, 16, BF, spare=4, seed=52)
    g = c.to_gpu()
    for shape in ((1, 2 ** 32 + 2, 1, 64), (1, 2, 2 ** 32 + 1, 64)):
        q = torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda").expand(shape)
        with pytest.raises(ValueError, match="too many"):
            ab.cache_score(g, q, per_token=False)
        with pytest.raises(ValueError, match="too many"):
            ab.cache_mass(g, q, torch.zeros(1, 2, 1, device="cuda"))
    k = torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda").expand(1, 1, 2 ** 32 + 1, 64)
    with pytest.raises(ValueError, match="too many"):
        ab.cache_append(g, k, k)


@pytest.mark.parametrize("T", [1, 16])  # the kernel for few rows, and that for many
@pytest.mark.parametrize("bad", [-1, 1000])
def test_mass_reports_counts_of_every_sequence(T, bad):
    c = HostCache([70, 300, 0, 200], 2, 64, 32, BF, seed=12)
    q, lse = c.randn(4, 4, T, 64).cuda(), 5 + torch.rand(4, 4, T, generator=c.g).cuda()
    for b in range(4):
        n = [T] * 4
        n[b] = bad
        for x, bits in ((n, ab.FLAG_BAD_INDEX), ([min(max(i, 0), T) for i in n], 0)):
            g, flag = c.to_gpu(), _flag()
            ab.cache_mass(g, q, lse, n_tok=_i32(*x), dev_flag=flag)
            assert ab.check_flag(flag) == bits, (b, x)
            if bits:
                got = g.mass
        assert torch.equal(got, g.mass)  # clamped


def _mass_of(c, q, lse, n_tok=None, plan=(None, None, None)):
    g = c.to_gpu()
    idx, cnt, w = (None if t is None else t.cuda() for t in plan)
    ab.cache_mass(g, q.cuda(), lse.cuda(), n_tok=n_tok, idx=idx, cnt=cnt, w=w)
    return g.mass.cpu()


@pytest.mark.parametrize("rows,T", [(1, 1), (1, 3), (3, 3)])  # a plan has one row, or one per token
@pytest.mark.parametrize("page,d", [(16, 64), (128, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_mass_outside_a_plan_takes_no_part(rows, T, page, d, bad):
    """NaN and infinity in the keys of a page that no row's plan has, and of slots below the new
    tokens in their page."""
    L = 3 * page + 9
    c = HostCache([L], 2, d, page, BF, seed=13)
    q, lse = c.randn(1, 4, T, d), 5 + torch.rand(1, 4, T, generator=c.g)
    idx = torch.full((1, 2, rows, c.max_pages), -1, dtype=torch.int32)
    idx[..., 0], idx[..., 1] = 0, 2
    cnt = torch.full((1, 2, rows), 2, dtype=torch.int32)
    plan = (idx, cnt, torch.full(idx.shape, 2.0))
    ref = _mass_of(c, q, lse, plan=plan)
    c.k[c.table[0, 1].long()] = bad
    c.k[c.table[0, 3].long(), :, : 9 - T] = bad
    assert torch.equal(_mass_of(c, q, lse, plan=plan), ref)


@pytest.mark.parametrize("G,T", [(1, 1), (3, 1), (3, 15), (5, 60)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_mass_of_infinite_keys(G, T, dtype):
    """A key whose logit is -inf for every row gets nothing; a row that saw nothing (its log-sum
    is -inf) and a row that does not exist add nothing, to a key whose logit is +inf or NaN for it
    either."""
    c = HostCache([500, 40], 1, 64, 64, dtype, seed=14)
    q, lse = c.randn(2, G, T, 64), 5 + torch.rand(2, G, T, generator=c.g)
    q[..., 0] = -q[..., 0].abs() - 1
    n_tok = _i32(T, max(1, min(T, 40) - 1))
    at = c.table[0, 2].long(), 0, 7
    c.mass[at] = 2.0
    ref = _mass_of(c, q, lse, n_tok)
    c.k[at] = 0
    c.k[at[0], 0, 7, 0] = math.inf
    got = _mass_of(c, q, lse, n_tok)
    assert float(got[at]) == 2.0
    got[at] = ref[at]
    assert torch.equal(got, ref)
    # rows that saw nothing
    lse[0, :, :] = -math.inf
    q[0, :, :, 0] *= -1
    c.k[at[0], 0, 7, 1] = math.nan
    got = _mass_of(c, q, lse, n_tok)
    assert torch.equal(got[c.table[0, :8].long()], c.mass[c.table[0, :8].long()])


@pytest.mark.parametrize("T,G", [(1, 2), (4, 4), (4, 10), (64, 3), (64, 5)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("L", [20, 3000])
def test_attn_nan_reaches_the_rows_that_see_it(T, G, dtype, L):
    """A NaN query gives a row of NaN with a NaN log-sum, however its keys are shared out; a NaN
    key gives that to the rows of its sequence and head. No other row changes."""
    c = HostCache([L, 200], 2, 64, 16, dtype, seed=18)
    q, k, v = (t.cuda() for t in (c.randn(2, 2 * G, T, 64), c.randn(2, 2, T, 64), c.randn(2, 2, T, 64)))
    out, lse = ab.cache_attn(c.to_gpu(), q, k, v, want_lse=True)
    bad = q.clone()
    bad[0, 1, T // 2] = math.nan
    got, got_lse = ab.cache_attn(c.to_gpu(), bad, k, v, want_lse=True)
    assert bool(got[0, 1, T // 2].isnan().all()) and bool(got_lse[0, 1, T // 2].isnan())
    got[0, 1, T // 2], got_lse[0, 1, T // 2] = out[0, 1, T // 2], lse[0, 1, T // 2]
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
    c.k[c.table[0, 1].long(), 0, :4] = math.nan
    c.k[c.table[0, 0].long(), 0] = math.nan  # a whole page, in a call on few keys all that a warp has
    got, got_lse = ab.cache_attn(c.to_gpu(), q, k, v, want_lse=True)
    assert bool(got[0, :G].isnan().all()) and bool(got_lse[0, :G].isnan().all())
    assert torch.equal(got[0, G:], out[0, G:]) and torch.equal(got[1], out[1])
    assert torch.equal(got_lse[0, G:], lse[0, G:]) and torch.equal(got_lse[1], lse[1])


@pytest.mark.parametrize("pages", [5, 700])
def test_score_nan_reaches_its_rows(pages):
    """NaN in pages' sums makes every share of the rows over them NaN, also where a whole CTA of a
    cluster has nothing else."""
    c = HostCache([16 * pages - 3], 2, 64, 16, BF, seed=19)
    q = c.randn(1, 4, 2, 64)
    for parts in (1, 2, 4, 8, 16):
        n = -(-pages // parts)
        for at in {0, min(n, pages - 1), n * ((pages - 1) // n)}:
            g = c.to_gpu()
            g.ksum[c.table[0, at : min(pages, at + n)].long().cuda(), 0] = math.nan
            got = ab.cache_score(g, q.cuda())
            assert bool(got[0, 0, :, :pages].isnan().all()) and not bool(got[0, 1].isnan().any()), (parts, at)


def test_handle_follows_its_tensors():
    """Tensors of a handle that are set to other memory (an offloaded cache that comes back, say)."""
    c = HostCache([100, 30], 2, 64, 32, BF, spare=4, seed=15)
    for b in range(2):
        c.allocate(b, 128)
    g, other = c.to_gpu(), c.to_gpu()
    old = {n: getattr(g, n).clone() for n in ("k", "v", "length", "ksum", "mass", "pos")}
    kept = [getattr(g, n).detach() for n in old]  # the first memory lives on
    for n in old:
        getattr(g, n).set_(getattr(other, n).clone())
    q, k, v = c.randn(2, 4, 1, 64).cuda(), c.randn(2, 2, 1, 64).cuda(), c.randn(2, 2, 1, 64).cuda()
    ab.cache_append(g, k, v)
    ab.cache_append(other, k, v)
    for n, t in zip(old, kept):
        assert torch.equal(t, old[n]), n
        assert torch.equal(getattr(g, n), getattr(other, n)), n
    g.length.set_(torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="length must be"):
        ab.cache_attn(g, q)
    g.k.set_(torch.empty(0, dtype=BF, device="cuda"))  # no pages to read
    with pytest.raises(ValueError, match="k must be"):
        ab.cache_append(g, k, v)


@pytest.mark.parametrize("Hk,G,T,d,page", [(2, 4, 20, 128, 32), (1, 5, 64, 64, 16), (2, 3, 90, 128, 128),
                                           (1, 24, 3, 64, 64)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("use", ["all", "plan"])
def test_tiles_read_nothing_behind_a_sequence(Hk, G, T, d, page, dtype, use):
    """The tensor-core kernels copy whole tiles: NaN in every row that no sequence owns and in
    tokens behind n_tok changes nothing."""
    c = HostCache([45, 100, 0, 7 * page + 3, 2 * page], Hk, d, page, dtype, spare=3, seed=16)
    B = c.B
    q, k, v = c.randn(B, Hk * G, T, d), c.randn(B, Hk, T, d), c.randn(B, Hk, T, d)
    n = [T, max(1, T - 1), 1, T // 2, 0]
    idx = torch.full((B, Hk, 1, c.max_pages), -1, dtype=torch.int32)
    idx[..., :3] = torch.tensor([0, 1, 7])  # the last pages of some, behind others
    cnt = torch.full((B, Hk, 1), 3, dtype=torch.int32)
    plan = (idx.cuda(), cnt.cuda()) if use == "plan" else (None, None)

    def run():
        g = c.to_gpu()
        out, lse = ab.cache_attn(g, q.cuda(), k.cuda(), v.cuda(), n_tok=_i32(*n), idx=plan[0], cnt=plan[1],
                                 want_lse=True)
        m = torch.full_like(g.mass, 7.0)
        ab.cache_mass(g, q.cuda(), lse, n_tok=_i32(*[min(a, int(b)) for a, b in zip(n, c.length)]), out=m)
        return out.cpu(), lse.cpu(), m.cpu()

    ref = run()
    owned = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b in range(B):
        s = torch.arange(int(c.length[b]))
        owned[c.table[b, s // page].long(), s % page] = True
    assert bool((~owned).any())
    for bad in (math.nan, math.inf):
        for t in (c.k, c.v):
            t.permute(0, 2, 1, 3)[~owned] = bad
        for b in range(B):
            for t in (k, v, q):
                t[b, :, n[b]:] = bad
        for a, e in zip(run(), ref):
            assert torch.equal(a, e) and not bool(a.isnan().any())


def test_readme_loop_keeps_the_newest_tokens():
    """README's generation loop, run as it stands past its first evictions."""
    with open(os.path.join(os.path.dirname(HERE), "README.md")) as f:
        text = f.read()
    text = text[text.index("# generation over a key/value cache"):]
    scope = {"torch": torch, "ab": ab}
    exec(text[: text.index("\n\n")], scope)
    c, next_pos = scope["c"], scope["next_pos"]
    assert c.length.tolist() == [4096, 4096] and next_pos.tolist() == [4106, 4106]
    for b in range(2):
        pos = c.pos[c.table[b, :32].long()].transpose(0, 1).reshape(8, 4096).sort(-1).values
        assert bool((pos[:, 1:] > pos[:, :-1]).all())  # no position twice
        assert torch.equal(pos[:, -64:], torch.arange(4106 - 64, 4106, device="cuda").int().expand(8, -1))


@pytest.mark.parametrize("T", [1, 12])
def test_generation_with_eviction_captured_and_replayed(T):
    """Append, mass, selection of the kept slots and their moves in one graph; two graphs that
    share a workspace, replayed in turn, give what eager calls give."""
    B, Hk, G, d, page, slots = 2, 2, 3, 64, 32, 200

    def fresh():
        c = HostCache([196, 150], Hk, d, page, FP, spare=16, max_pages=8, seed=23)
        for b in range(B):
            c.allocate(b, 8 * page)
        c.mass.zero_()
        return c, c.to_gpu()
    c, a = fresh()
    e = fresh()[1]
    toks = [[c.randn(B, h, T, d).cuda() for h in (Hk * G, Hk, Hk)] for _ in range(6)]
    bufs = [[torch.zeros_like(t) for t in toks[0]] for _ in range(2)]
    size = ab.cache_attn_workspace_bytes(a, Hk * G, T, False)
    ws, kws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (size, 4 * B * Hk * slots))

    def step(cache, q, k, v, next_pos):
        out, lse = ab.cache_attn(cache, q, k, v, want_lse=True, workspace=ws)
        ab.cache_append(cache, k, v, pos=next_pos)
        next_pos += T
        ab.cache_mass(cache, q, lse)
        src, n = ab.cache_keep(cache, slots, recent=2 * T, next_pos=next_pos, workspace=kws)
        ab.cache_compact(cache, src, n)
        return out, src, n

    pa, pe = a.length.clone(), e.length.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(fresh()[1], *bufs[0], pa.clone())
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in bufs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(step(a, *x, pa))
    torch.cuda.synchronize()
    for i, t in enumerate(toks):
        for dst, x in zip(bufs[i % 2], t):
            dst.copy_(x)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for x, y in zip(outs[i % 2], step(e, *t, pe)):
            assert torch.equal(x, y)
        for x in ("k", "v", "ksum", "mass", "pos", "length"):
            assert torch.equal(getattr(a, x), getattr(e, x)), x
    assert torch.equal(pa, pe) and a.length[0] == slots


def _check(got, lse, ref, dtype):
    out, ref_lse, tol, tol_lse = (x.cuda() for x in ref)
    err = (got.to(F64) - out).abs()
    assert bool((err <= tol + torch.finfo(dtype).eps / 2 * (out.abs() + tol) + 1e-7).all()), float(err.max())
    assert bool(((lse.to(F64) - ref_lse).abs() <= tol_lse + 2.0 ** -23 * ref_lse.abs()).all())


@pytest.mark.parametrize("T,G", [(1, 2), (9, 2), (20, 4), (64, 5), (100, 2)])
@pytest.mark.parametrize("how", ["heads", "batch", "tokens", "all"])
def test_attn_of_expanded_tokens(T, G, how):
    """New tokens whose keys and values are one row seen as many (strides of 0: no tensor map)."""
    c = HostCache([70, 0, 200], 2, 64, 32, BF, seed=24)
    q, k, v = c.randn(3, 2 * G, T, 64), c.randn(3, 2, T, 64), c.randn(3, 2, T, 64)
    cut = {"heads": (slice(None), slice(0, 1)), "batch": (slice(0, 1),), "all": (slice(0, 1),) * 3,
           "tokens": (slice(None), slice(None), slice(0, 1))}[how]
    k, v = (t[cut].expand(3, 2, T, 64) for t in (k, v))
    kg, vg = (t[cut].cuda().expand(3, 2, T, 64) for t in (k, v))
    qg = q[:1].cuda().expand(3, -1, -1, -1)
    n = torch.tensor([T, max(1, T - 3), T // 2])
    got, lse = ab.cache_attn(c.to_gpu(), qg, kg, vg, n_tok=n.int().cuda(), want_lse=True)
    _check(got, lse, attn(c, q[:1].expand(3, -1, -1, -1), k, v, n), BF)


@pytest.mark.parametrize("T,G", [(1, 1), (20, 1), (70, 5)])
@pytest.mark.parametrize("page,d", [(16, 128), (128, 64)])
def test_pool_of_one_page_and_one_head(T, G, page, d):
    """Dimensions of one element, whose strides mean nothing."""
    c = HostCache([page - 3], 1, d, page, FP, seed=25, max_pages=1)
    used = int(c.table[0, 0])
    c.k, c.v, c.mass, c.n_pages = c.k[used : used + 1], c.v[used : used + 1], c.mass[used : used + 1] * 0, 1
    c.pos, c.ksum = c.pos[:1], c.ksum[:1]
    c.table[0, 0] = 0
    g = c.to_gpu()
    q, k, v = c.randn(1, G, T, d), c.randn(1, 1, T, d), c.randn(1, 1, T, d)
    got, lse = ab.cache_attn(g, q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check(got, lse, attn(c, q, k, v), FP)
    n = min(T, page - 3)
    ab.cache_mass(g, q.cuda(), lse, n_tok=_i32(n))
    ref, tol = mass(c, q, lse.cpu(), [n])
    assert bool(((g.mass.cpu().to(F64) - ref).abs() <= tol + 1e-7).all())


@pytest.mark.parametrize("T", [1, 40])
def test_keys_and_values_side_by_side(T):
    """Keys and values in one buffer [n_pages, page, 2, Hk, d], other pages of it in use elsewhere."""
    c = HostCache([333, 64, 7], 3, 128, 64, BF, spare=5, seed=26)
    for b in range(3):
        c.allocate(b, int(c.length[b]) + T)
    buf = torch.full((c.n_pages + 2, 64, 2, 3, 128), math.nan, dtype=BF, device="cuda")
    k, v = (buf[1:-1, :, i].transpose(1, 2) for i in range(2))
    k.copy_(c.k)
    v.copy_(c.v)
    g = ab.KVCache(k=k, v=v, table=c.table.cuda(), length=c.length.cuda(), ksum=c.ksum.cuda(),
                   mass=torch.zeros(c.n_pages, 3, 64, device="cuda"))
    q, kn, vn = c.randn(3, 6, T, 128), c.randn(3, 3, T, 128), c.randn(3, 3, T, 128)
    got, lse = ab.cache_attn(g, q.cuda(), kn.cuda(), vn.cuda(), want_lse=True)
    _check(got, lse, attn(c, q, kn, vn), BF)
    ab.cache_append(g, kn.cuda(), vn.cuda())
    for b in range(3):
        s = torch.arange(int(c.length[b]), int(c.length[b]) + T)
        at = (c.table[b, s // 64].long(), slice(None), s % 64)
        c.k[at], c.v[at] = kn[b].transpose(0, 1), vn[b].transpose(0, 1)
    assert torch.equal(k.cpu(), c.k) and torch.equal(v.cpu(), c.v)
    assert bool(buf[0].isnan().all()) and bool(buf[-1].isnan().all())
    c.length += T
    c.mass.zero_()
    ab.cache_mass(g, q.cuda(), lse)
    ref, tol = mass(c, q, lse.cpu())
    assert bool(((g.mass.cpu().to(F64) - ref).abs() <= tol + 1e-7).all())
