"""Host-side checks of the key/value cache calls: every refusal that include/ab_attn.h
documents comes back synchronously with its status code, before anything is launched, so
this runs without a GPU. No pointer below is ever dereferenced."""

import ctypes

import pytest
import torch

import block_sparse_attention_ab_b200 as ab
from block_sparse_attention_ab_b200 import build
from block_sparse_attention_ab_b200.cache import AB_BF16, AB_F16, AB_F32, CacheStruct, TokensStruct

P = 0x10000
ODD = 0x10002
NULL, SHAPE, DTYPE, UNSUPPORTED, RANGE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 9, 10


@pytest.fixture(scope="module")
def L():
    build.build()
    return ab.lib()


def cache(**kw):
    f = dict(k=P, v=P, ksum=P, mass=P, pos=P, table=P, length=P, k_page=8192, k_head=4096, k_row=64,
             v_page=8192, v_head=4096, v_row=64, B=3, Hk=2, d=64, page=64, n_pages=10, max_pages=5, dtype=AB_BF16)
    f.update(kw)
    return CacheStruct(*(f[n] for n, _ in CacheStruct._fields_))


def tokens(p=P, sb=512, sh=256, st=64):
    return TokensStruct(p, sb, sh, st)


def append(L, c, k=None, v=None, T=4, n_new=P, sel=P, start=P + 4096, pos0=P):
    return L.ab_cache_append(c, k or tokens(), v or tokens(), T, n_new, sel, start, pos0, None, None)


def score(L, c, q=None, Hq=4, T=4, n_tok=P, per_token=1, first=0, recent=0, scores=P):
    return L.ab_cache_score(c, q or tokens(), Hq, T, n_tok, per_token, first, recent, scores, None, None)


def attn(L, c, q=None, k=None, v=None, Hq=4, T=4, idx=P, cnt=P, w=P, per_token=0, out=P, out_dtype=AB_BF16, lse=P,
         ws=P, ws_bytes=1 << 40):
    return L.ab_cache_attn(c, q or tokens(), k or tokens(), v or tokens(), Hq, T, P, P, idx, cnt, w, per_token, out,
                           out_dtype, lse, ws, ws_bytes, None, None)


def mass(L, c, q=None, Hq=4, T=4, lse=P, idx=None, cnt=None, w=None, per_token=0, out=None):
    return L.ab_cache_mass(c, q or tokens(), Hq, T, P, P, lse, idx, cnt, w, per_token, out, None, None)


def keep(L, c, budget=100, recent=0, next_pos=P, score=None, pos=None, src=P, n_keep=P, ws=P, ws_bytes=1 << 40):
    return L.ab_cache_keep(c, budget, recent, next_pos, score, pos, None, src, n_keep, ws, ws_bytes, None, None)


def compact(L, c, budget=100, src=P, n_keep=P + 4096):
    return L.ab_cache_compact(c, budget, src, n_keep, None, None)


CALLS = [append, score, attn, mass, keep, compact]
PAGES = [append, attn, mass, compact]  # these read or write the pages


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,code", [
    (dict(table=None), NULL), (dict(length=None), NULL),
    (dict(B=0), SHAPE), (dict(Hk=-1), SHAPE), (dict(n_pages=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(dtype=AB_F32), DTYPE), (dict(dtype=7), DTYPE),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED),
    (dict(B=65536), RANGE), (dict(Hk=65536), RANGE), (dict(B=2000, Hk=2000), RANGE), (dict(max_pages=1 << 25), RANGE),
    (dict(table=ODD), ALIGN), (dict(length=ODD), ALIGN), (dict(ksum=P + 8), ALIGN), (dict(mass=ODD), ALIGN),
    (dict(pos=ODD), ALIGN),
])
def test_cache_refusals(L, call, bad, code):
    assert call(L, cache(**bad)) == code


@pytest.mark.parametrize("call", PAGES)
@pytest.mark.parametrize("bad,code", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(k_row=68), ALIGN), (dict(k_head=4), ALIGN), (dict(v_page=8190), ALIGN), (dict(v_row=-64), ALIGN),
    (dict(k_page=1 << 40), ALIGN),
])
def test_page_refusals(L, call, bad, code):
    assert call(L, cache(**bad)) == code


def test_token_refusals(L):
    c = cache()
    for bad in (dict(p=P + 8), dict(st=60), dict(sh=-256), dict(sb=4)):
        t = tokens(**bad)
        assert append(L, c, k=t) == ALIGN and append(L, c, v=t) == ALIGN
        assert attn(L, c, q=t) == ALIGN and attn(L, c, k=t) == ALIGN and attn(L, c, v=t) == ALIGN
        assert score(L, c, q=t) == ALIGN and mass(L, c, q=t) == ALIGN
    none = tokens(p=None)
    assert append(L, c, k=none) == NULL and append(L, c, v=none) == NULL
    assert attn(L, c, q=none) == NULL and score(L, c, q=none) == NULL and mass(L, c, q=none) == NULL
    assert attn(L, c, k=none) == NULL  # k without v
    assert append(L, c, T=0) == SHAPE and append(L, c, T=(1 << 20) + 1) == RANGE
    for call in (score, attn, mass):
        assert call(L, c, Hq=3) == SHAPE and call(L, c, Hq=0) == SHAPE and call(L, c, T=0) == SHAPE
        assert call(L, c, T=129) == RANGE and call(L, c, Hq=4098 * 2) == RANGE


def test_argument_refusals(L):
    c = cache()
    assert append(L, c, start=P) == UNSUPPORTED  # the cache's own length array
    assert append(L, c, n_new=ODD) == ALIGN and append(L, c, sel=ODD) == ALIGN
    assert score(L, cache(ksum=None)) == NULL and score(L, c, scores=None) == NULL
    assert score(L, c, first=-1) == RANGE and score(L, c, recent=-1) == RANGE
    assert score(L, cache(max_pages=65537, page=16)) == RANGE
    assert attn(L, c, out=None) == NULL and attn(L, c, out=P + 8) == ALIGN
    assert attn(L, c, cnt=None) == NULL and attn(L, c, idx=None, cnt=None) == NULL
    assert attn(L, c, idx=None, cnt=None, w=None, per_token=1) == NULL
    assert attn(L, c, out_dtype=AB_F16) == DTYPE and attn(L, cache(dtype=AB_F16)) == DTYPE
    assert attn(L, c, ws=None) == WORKSPACE and attn(L, c, ws_bytes=64) == WORKSPACE
    assert mass(L, cache(mass=None)) == NULL and mass(L, c, lse=None) == NULL
    assert mass(L, c, idx=P) == NULL and mass(L, c, per_token=1) == NULL
    assert keep(L, c, budget=0) == RANGE and keep(L, c, recent=-1) == RANGE
    assert keep(L, cache(mass=None)) == NULL and keep(L, c, recent=1, next_pos=None) == NULL
    assert keep(L, cache(pos=None), recent=1) == NULL
    assert keep(L, c, src=None) == NULL and keep(L, c, n_keep=None) == NULL
    assert keep(L, c, ws=None) == WORKSPACE and keep(L, c, ws_bytes=100) == WORKSPACE
    assert compact(L, c, budget=0) == RANGE and compact(L, c, src=None) == NULL
    assert compact(L, c, n_keep=P) == UNSUPPORTED  # the cache's own length array


def test_workspace_sizes(L):
    n = ctypes.c_size_t(1)
    c = cache(d=128, B=4, Hk=8)
    small = None
    for T in (1, 4, 64, 128):
        for per_token in (0, 1):
            assert L.ab_cache_attn_workspace_size(c, 40, T, per_token, ctypes.byref(n)) == 0
            assert 0 < n.value < 400 << 20  # a few hundred MB at most, whatever the shape
            small = small or n.value
    assert small < 16 << 20
    assert L.ab_cache_attn_workspace_size(c, 40, 0, 0, ctypes.byref(n)) == SHAPE and n.value == 0
    assert L.ab_cache_attn_workspace_size(c, 40, 4, 0, None) == NULL
    assert L.ab_cache_keep_workspace_size(c, 1000, ctypes.byref(n)) == 0 and n.value == 4 * 4 * 8 * 1000
    assert L.ab_cache_keep_workspace_size(c, 0, ctypes.byref(n)) == RANGE and n.value == 0


def test_binding_refuses_host_tensors():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, length = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        ab.KVCache(k=k, v=k, table=table, length=length)
    with pytest.raises(TypeError, match="must be a tensor"):
        ab.KVCache(k=k, v=None, table=table, length=length)


def test_new_flag_bit_is_its_own():
    bits = [ab.FLAG_BAD_SCORE, ab.FLAG_BAD_INDEX, ab.FLAG_BAD_WEIGHT, ab.FLAG_TIMEOUT, ab.FLAG_SCHED_COLLISION,
            ab.FLAG_CACHE_FULL]
    assert bits == [1, 2, 4, 8, 16, 32]


def test_append_refuses_arrays_in_the_length_it_writes(L):
    """With start, length is written while the other arrays are read; parts of it too."""
    c = cache(length=P + 4096)  # B = 3: 12 bytes
    far = dict(n_new=P, sel=P + 64, start=P + 256, pos0=P + 512)
    for name in far:
        for at in (P + 4096, P + 4100, P + 4104, P + 4088):
            assert append(L, c, **{**far, name: at}) == UNSUPPORTED, (name, at)
    # at the sequence's end a second kernel reads n_new and writes length, each at its sequence
    assert append(L, c, **{**far, "start": None, "n_new": P + 4100}) == UNSUPPORTED


def test_keep_refuses_outputs_over_its_inputs(L):
    """n_keep and src are written by one head while the others read length and next_pos."""
    c = cache(length=P + 4096)  # B = 3, Hk = 2: src has 600 words
    far = dict(src=P + 32768, n_keep=P + 65536, next_pos=P + 8192, recent=1)
    for at in (P + 4096, P + 4100, P + 4088, P + 8192, P + 8200):
        assert keep(L, c, **{**far, "n_keep": at}) == UNSUPPORTED
    for at in (P + 4096, P + 4096 - 2396, P + 8200, P + 8192 - 4):
        assert keep(L, c, **{**far, "src": at}) == UNSUPPORTED
    # the length given in place of the cache's
    assert L.ab_cache_keep(c, 100, 0, None, None, None, P + 65536, P + 32768, P + 65540, P, 1 << 40, None, None) == \
        UNSUPPORTED


def test_compact_refuses_arrays_in_the_length_it_writes(L):
    c = cache(length=P + 4096)  # B = 3
    for at in (P + 4096, P + 4104, P + 4088):
        assert compact(L, c, src=P + 32768, n_keep=at) == UNSUPPORTED
    for at in (P + 4096, P + 4104, P + 4096 - 2396):
        assert compact(L, c, src=at, n_keep=P + 65536) == UNSUPPORTED
