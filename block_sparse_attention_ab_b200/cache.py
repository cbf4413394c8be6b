"""Key/value cache: generation token by token over the keys and values of earlier steps.

Binding of the ab_cache_* calls of ``include/ab_attn.h`` (compiled: csrc/cache_bind.cpp). One
serving step over a cache, with block-sparse attention and a bounded number of slots:

  scores = cache_score(c, q)                       # cheap page scores for the new tokens
  idx, cnt, w = select(scores, budget, "sip")      # the pages to read
  out, lse = cache_attn(c, q, k, v, idx=idx, cnt=cnt, w=w, want_lse=True)
  cache_append(c, k, v, pos=next_pos)              # (sel=: the accepted tokens of a tree)
  next_pos += 1                                    # by the tokens appended; evictions change nothing
  cache_mass(c, q, lse, idx=idx, cnt=cnt, w=w)     # the weight every slot received
  src, n = cache_keep(c, slots, recent=64, next_pos=next_pos)
  cache_compact(c, src, n)                         # evict down to `slots`

Without a plan cache_attn reads the whole cache. q is [B, Hq, T, d] and k, v are
[B, Hk, T, d], in any strides that keep rows contiguous and 16-byte aligned.
"""

from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

AB_F32, AB_BF16, AB_F16 = 0, 1, 2
MAX_TREE = 128  # AB_MAX_TREE: new tokens per sequence of cache_attn, cache_score, cache_mass
FLAG_CACHE_FULL = 32
_I64, _I32, _P = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class CacheStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "ksum", "mass", "pos", "table", "length")] + \
               [(n, _I64) for n in ("k_page", "k_head", "k_row", "v_page", "v_head", "v_row")] + \
               [(n, _I32) for n in ("B", "Hk", "d", "page", "n_pages", "max_pages", "dtype")]


class TokensStruct(ctypes.Structure):
    _fields_ = [("p", _P), ("sb", _I64), ("sh", _I64), ("st", _I64)]


def bind(L):
    """Argument types of the ab_cache_* calls, for ctypes (the functions below go through the
    compiled binding)."""
    C, T, I, P, Z = CacheStruct, TokensStruct, ctypes.c_int, _P, ctypes.c_size_t
    size_p = ctypes.POINTER(ctypes.c_size_t)
    for name, args in {
        "ab_cache_append": [C, T, T, I, P, P, P, P, P, P],
        "ab_cache_score": [C, T, I, I, P, I, I, I, P, P, P],
        "ab_cache_attn_workspace_size": [C, I, I, I, size_p],
        "ab_cache_attn": [C, T, T, T, I, I, P, P, P, P, P, I, P, I, P, P, Z, P, P],
        "ab_cache_mass": [C, T, I, I, P, P, P, P, P, P, I, P, P, P],
        "ab_cache_keep_workspace_size": [C, I, size_p],
        "ab_cache_keep": [C, I, I, P, P, P, P, P, P, P, Z, P, P],
        "ab_cache_compact": [C, I, P, P, P, P],
    }.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_binding = None


def _load():
    """The compiled binding (raises if it was not built)."""
    global _binding
    if _binding is None:
        from . import AbError, lib
        lib()
        from . import _cache_bind
        _cache_bind.set_error(AbError)
        _binding = _cache_bind
    return _binding


@dataclasses.dataclass(frozen=True, eq=False)
class KVCache:
    """Pages k, v [n_pages, Hk, page, d] (bf16 or fp16, any strides with contiguous rows),
    table int32 [B, max_pages], length int32 [B]; optional ksum fp32 [n_pages, Hk, d] (for
    cache_score), mass fp32 and pos int32 [n_pages, Hk, page] (for eviction). The tensors
    are the caller's; the calls write into them."""

    k: torch.Tensor
    v: torch.Tensor
    table: torch.Tensor
    length: torch.Tensor
    ksum: Optional[torch.Tensor] = None
    mass: Optional[torch.Tensor] = None
    pos: Optional[torch.Tensor] = None

    def __post_init__(self):
        for name in ("k", "v", "table", "length"):
            if not isinstance(getattr(self, name), torch.Tensor):
                raise TypeError(f"{name} must be a tensor")
        for name in ("k", "v"):
            if not getattr(self, name).is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor")
        object.__setattr__(self, "_c", _load().Cache(self.k, self.v, self.table, self.length, self.ksum,
                                                     self.mass, self.pos))


def make_cache(B: int, Hk: int, d: int, n_pages: int, max_pages: int, page: int = 128,
               dtype=torch.bfloat16, device="cuda", sums: bool = True, masses: bool = True) -> KVCache:
    """An empty cache of n_pages pages. Its table is the caller's to fill: table[b, i] is the
    pool page of sequence b's i-th page (-1 here: none)."""
    def new(*shape, dt, fill=0):
        return torch.full(shape, fill, dtype=dt, device=device)
    return KVCache(k=new(n_pages, Hk, page, d, dt=dtype), v=new(n_pages, Hk, page, d, dt=dtype),
                   table=new(B, max_pages, dt=torch.int32, fill=-1), length=new(B, dt=torch.int32),
                   ksum=new(n_pages, Hk, d, dt=torch.float32) if sums else None,
                   mass=new(n_pages, Hk, page, dt=torch.float32) if masses else None,
                   pos=new(n_pages, Hk, page, dt=torch.int32) if masses else None)


def cache_append(cache: KVCache, k, v, n_new=None, sel=None, start=None, pos=None, dev_flag=None):
    """Write new tokens' keys and values (rows sel[b, i] of k and v [B, Hk, T, d], or rows
    0 .. n_new[b] - 1) at slot start[b] (default: the sequence's end) and set length. pos int32
    [B]: the first new token's position (default: its slot, which is its position only while
    nothing has been evicted). With start, no array may lie in cache.length, which the call
    writes; give clones of it."""
    cache._c.append(k, v, n_new, sel, start, pos, dev_flag)


def cache_score(cache: KVCache, q, n_tok=None, per_token: bool = True, first: int = 0, recent: int = 0,
                out=None, dev_flag=None):
    """Page scores fp32 [B, Hk, T or 1, max_pages] of the tokens q [B, Hq, T, d], for select().
    The first `first` and last `recent` pages score 2: they are always kept. cache_compact moves
    the newest tokens into holes anywhere, so after an eviction the last pages are not the newest
    tokens' any more."""
    return cache._c.score(q, n_tok, per_token, first, recent, out, dev_flag)


def cache_attn_workspace_bytes(cache: KVCache, Hq: int, T: int, per_token: bool) -> int:
    return cache._c.attn_workspace(Hq, T, per_token)


def cache_attn(cache: KVCache, q, k=None, v=None, n_tok=None, tree=None, idx=None, cnt=None, w=None,
               want_lse: bool = False, out=None, out_dtype=None, workspace=None, dev_flag=None):
    """Attention of the new tokens q [B, Hq, T, d] over the cache (whole, or the pages of a
    plan) and over the new tokens' own k, v [B, Hk, T, d] where tree [B, T, T] (bool; default:
    earlier tokens and the token itself) allows. Returns out [B, Hq, T, d] [and lse]."""
    return cache._c.attn(q, k, v, n_tok, tree, idx, cnt, w, want_lse, out, out_dtype, workspace, dev_flag)


def cache_mass(cache: KVCache, q, lse, n_tok=None, sel=None, idx=None, cnt=None, w=None, out=None,
               dev_flag=None):
    """Add to the cache's mass (or write to `out`, like it, mass plus) the weight that every
    slot got from a sequence's last n_tok[b] tokens, which have been appended: rows sel[b, i]
    (or i) of cache_attn's q and lse. Returns the tensor written."""
    return cache._c.mass(q, lse, n_tok, sel, idx, cnt, w, out, dev_flag)


def cache_keep(cache: KVCache, budget: int, recent: int = 0, next_pos=None, score=None, pos=None,
               length=None, workspace=None, dev_flag=None):
    """The slots a cache of `budget` slots keeps, per sequence and key head: (src int32
    [B, Hk, budget], n_keep int32 [B]) for cache_compact. Slots with pos >= next_pos[b] - recent
    stay first, then those of the largest score (default: the cache's mass)."""
    return cache._c.keep(budget, recent, next_pos, score, pos, length, workspace, dev_flag)


def cache_compact(cache: KVCache, src, n_keep, dev_flag=None):
    """Carry out cache_keep's moves and set length to n_keep."""
    cache._c.compact(src, n_keep, dev_flag)
