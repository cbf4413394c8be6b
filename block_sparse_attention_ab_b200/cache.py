"""Key/value cache: generation token by token over the keys and values of earlier steps.

Thin binding of the ab_cache_* calls of ``include/ab_attn.h``. One serving step over a
cache, with block-sparse attention and a bounded number of slots:

  scores = cache_score(c, q)                       # cheap page scores for the new tokens
  idx, cnt, w = select(scores, budget, "sip")      # the pages to read
  out, lse = cache_attn(c, q, k, v, idx=idx, cnt=cnt, w=w, want_lse=True)
  cache_append(c, k, v)                            # (sel=: the accepted tokens of a tree)
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
_CODES = {torch.bfloat16: AB_BF16, torch.float16: AB_F16}
_I64, _I32, _P = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class CacheStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "ksum", "mass", "pos", "table", "length")] + \
               [(n, _I64) for n in ("k_page", "k_head", "k_row", "v_page", "v_head", "v_row")] + \
               [(n, _I32) for n in ("B", "Hk", "d", "page", "n_pages", "max_pages", "dtype")]


class TokensStruct(ctypes.Structure):
    _fields_ = [("p", _P), ("sb", _I64), ("sh", _I64), ("st", _I64)]


_NO_TOKENS = TokensStruct(None, 0, 0, 0)


def bind(L):
    """Argument types of the ab_cache_* calls."""
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


def _lib():
    from . import lib
    return lib()


def _call(cache, name, *args):
    """Run a library call on the current stream of the cache's device."""
    from . import _check
    f = getattr(_lib(), name)
    dev = cache.k.device
    if torch.cuda.current_device() == dev.index:
        code = f(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = f(*args, torch.cuda.current_stream().cuda_stream)
    _check(code, name)


def _arr(t, dtype, shape, cache, name):
    """Data pointer of a contiguous tensor on the cache's device (None stays None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != cache.k.device:
        raise ValueError(f"{name} must be on {cache.k.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _flag(t, cache):
    return None if t is None else _arr(t, torch.int32, (1,), cache, "dev_flag")


def _tokens(t, cache, heads, name):
    if not isinstance(t, torch.Tensor) or t.dtype != cache.k.dtype:
        raise TypeError(f"{name} must be a {cache.k.dtype} tensor")
    if t.device != cache.k.device:
        raise ValueError(f"{name} must be on {cache.k.device}")
    if t.dim() != 4 or t.shape[0] != cache.B or t.shape[3] != cache.d or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{cache.B}, {heads or 'Hq'}, T, {cache.d}], got {tuple(t.shape)}")
    sb, sh, st, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # the stride of a dimension of one element is never used
    B, H, T = t.shape[:3]
    return TokensStruct(t.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, st if T > 1 else 0)


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
        k, v = self.k, self.v
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dtype not in _CODES:
                raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name} must be [n_pages, Hk, page, d] with contiguous rows")
        if v.dtype != k.dtype or v.shape != k.shape or v.device != k.device:
            raise ValueError("k and v must have one shape, type and device")
        if self.table.dim() != 2:
            raise ValueError("table must be [B, max_pages]")
        n_pages, Hk, page, d = k.shape
        B, max_pages = self.table.shape
        s = CacheStruct(
            k.data_ptr(), v.data_ptr(),
            _arr(self.ksum, torch.float32, (n_pages, Hk, d), self, "ksum"),
            _arr(self.mass, torch.float32, (n_pages, Hk, page), self, "mass"),
            _arr(self.pos, torch.int32, (n_pages, Hk, page), self, "pos"),
            _arr(self.table, torch.int32, (B, max_pages), self, "table"),
            _arr(self.length, torch.int32, (B,), self, "length"),
            *(t.stride(i) if t.shape[i] > 1 else 0 for t in (k, v) for i in range(3)),
            B, Hk, d, page, n_pages, max_pages, _CODES[k.dtype])
        object.__setattr__(self, "B", B)
        object.__setattr__(self, "Hk", Hk)
        object.__setattr__(self, "page", page)
        object.__setattr__(self, "d", d)
        object.__setattr__(self, "max_pages", max_pages)
        object.__setattr__(self, "struct", s)
        object.__setattr__(self, "_sizes", {})  # workspace bytes by call shape


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
    [B]: the first new token's position (default: its slot)."""
    T = k.shape[2]
    B = cache.B
    tk, tv = _tokens(k, cache, cache.Hk, "k"), _tokens(v, cache, cache.Hk, "v")
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    _call(cache, "ab_cache_append", cache.struct, tk, tv, T,
          _arr(n_new, torch.int32, (B,), cache, "n_new"), _arr(sel, torch.int32, (B, T), cache, "sel"),
          _arr(start, torch.int32, (B,), cache, "start"), _arr(pos, torch.int32, (B,), cache, "pos"),
          _flag(dev_flag, cache))


def cache_score(cache: KVCache, q, n_tok=None, per_token: bool = True, first: int = 0, recent: int = 0,
                out=None, dev_flag=None):
    """Page scores fp32 [B, Hk, T or 1, max_pages] of the tokens q [B, Hq, T, d], for select()."""
    tq = _tokens(q, cache, None, "q")
    Hq, T = q.shape[1:3]
    shape = (cache.B, cache.Hk, T if per_token else 1, cache.max_pages)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=q.device)
    _call(cache, "ab_cache_score", cache.struct, tq, Hq, T, _arr(n_tok, torch.int32, (cache.B,), cache, "n_tok"),
          int(bool(per_token)), first, recent, _arr(out, torch.float32, shape, cache, "out"),
          _flag(dev_flag, cache))
    return out


def cache_attn_workspace_bytes(cache: KVCache, Hq: int, T: int, per_token: bool) -> int:
    key = (Hq, T, per_token)
    if key not in cache._sizes:
        from . import _check
        n = ctypes.c_size_t(0)
        _check(_lib().ab_cache_attn_workspace_size(cache.struct, Hq, T, int(per_token), ctypes.byref(n)),
               "ab_cache_attn_workspace_size")
        cache._sizes[key] = n.value
    return cache._sizes[key]


def _plan(cache, T, idx, cnt, w):
    """Pointers of a plan and whether it has a row per token."""
    if idx is None:
        if cnt is not None or w is not None:
            raise ValueError("cnt and w go with idx")
        return None, None, None, 0
    if cnt is None:
        raise ValueError("idx needs cnt")
    Tp = idx.shape[2] if idx.dim() == 4 else -1
    if Tp not in (1, T):
        raise ValueError(f"idx must have 1 or {T} rows per key head")
    rows = (cache.B, cache.Hk, Tp)
    return (_arr(idx, torch.int32, rows + (cache.max_pages,), cache, "idx"),
            _arr(cnt, torch.int32, rows, cache, "cnt"),
            _arr(w, torch.float32, rows + (cache.max_pages,), cache, "w"), int(Tp == T))


def cache_attn(cache: KVCache, q, k=None, v=None, n_tok=None, tree=None, idx=None, cnt=None, w=None,
               want_lse: bool = False, out=None, out_dtype=None, workspace=None, dev_flag=None):
    """Attention of the new tokens q [B, Hq, T, d] over the cache (whole, or the pages of a
    plan) and over the new tokens' own k, v [B, Hk, T, d] where tree [B, T, T] (bool; default:
    earlier tokens and the token itself) allows. Returns out [B, Hq, T, d] [and lse]."""
    tq = _tokens(q, cache, None, "q")
    B, Hq, T, d = q.shape
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    tk = tv = _NO_TOKENS
    if k is not None:
        tk, tv = _tokens(k, cache, cache.Hk, "k"), _tokens(v, cache, cache.Hk, "v")
        if k.shape[2] != T or v.shape[2] != T:
            raise ValueError("q, k and v must have the same number of tokens")
    pi, pc, pw, per_token = _plan(cache, T, idx, cnt, w)
    if out_dtype is None:
        out_dtype = q.dtype if out is None else out.dtype
    if out_dtype is not q.dtype and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be {q.dtype} or torch.float32")
    if out is None:
        out = torch.empty((B, Hq, T, d), dtype=out_dtype, device=q.device)
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device) if want_lse else None
    if workspace is None:
        workspace = torch.empty(cache_attn_workspace_bytes(cache, Hq, T, bool(per_token)), dtype=torch.uint8,
                                device=q.device)
    _call(cache, "ab_cache_attn", cache.struct, tq, tk, tv, Hq, T, _arr(n_tok, torch.int32, (B,), cache, "n_tok"),
          _arr(tree, torch.bool, (B, T, T), cache, "tree"), pi, pc, pw, per_token,
          _arr(out, out_dtype, (B, Hq, T, d), cache, "out"), _CODES.get(out_dtype, AB_F32),
          None if lse is None else lse.data_ptr(),
          _arr(workspace, torch.uint8, tuple(workspace.shape), cache, "workspace"), workspace.numel(),
          _flag(dev_flag, cache))
    return (out, lse) if want_lse else out


def cache_mass(cache: KVCache, q, lse, n_tok=None, sel=None, idx=None, cnt=None, w=None, out=None,
               dev_flag=None):
    """Add to the cache's mass (or write to `out`, like it, mass plus) the weight that every
    slot got from a sequence's last n_tok[b] tokens, which have been appended: rows sel[b, i]
    (or i) of cache_attn's q and lse. Returns the tensor written."""
    tq = _tokens(q, cache, None, "q")
    B, Hq, T = q.shape[:3]
    if cache.mass is None:
        raise ValueError("the cache has no mass")
    pi, pc, pw, per_token = _plan(cache, T, idx, cnt, w)
    _call(cache, "ab_cache_mass", cache.struct, tq, Hq, T, _arr(n_tok, torch.int32, (B,), cache, "n_tok"),
          _arr(sel, torch.int32, (B, T), cache, "sel"), _arr(lse, torch.float32, (B, Hq, T), cache, "lse"),
          pi, pc, pw, per_token, _arr(out, torch.float32, tuple(cache.mass.shape), cache, "out"),
          _flag(dev_flag, cache))
    return cache.mass if out is None else out


def cache_keep(cache: KVCache, budget: int, recent: int = 0, next_pos=None, score=None, pos=None,
               length=None, workspace=None, dev_flag=None):
    """The slots a cache of `budget` slots keeps, per sequence and key head: (src int32
    [B, Hk, budget], n_keep int32 [B]) for cache_compact. Slots with pos >= next_pos[b] - recent
    stay first, then those of the largest score (default: the cache's mass)."""
    c, B = cache, cache.B
    slots = (c.k.shape[0], c.Hk, c.page)
    budget = int(budget)
    src = torch.empty((B, c.Hk, max(budget, 0)), dtype=torch.int32, device=c.k.device)
    n_keep = torch.empty((B,), dtype=torch.int32, device=c.k.device)
    if workspace is None:  # ab_cache_keep_workspace_size: one int32 per (sequence, key head, slot)
        workspace = torch.empty((B * c.Hk * max(budget, 1) * 4,), dtype=torch.uint8, device=c.k.device)
    _call(c, "ab_cache_keep", c.struct, budget, int(recent), _arr(next_pos, torch.int32, (B,), c, "next_pos"),
          _arr(score, torch.float32, slots, c, "score"), _arr(pos, torch.int32, slots, c, "pos"),
          _arr(length, torch.int32, (B,), c, "length"), src.data_ptr(), n_keep.data_ptr(),
          _arr(workspace, torch.uint8, tuple(workspace.shape), c, "workspace"), workspace.numel(),
          _flag(dev_flag, c))
    return src, n_keep


def cache_compact(cache: KVCache, src, n_keep, dev_flag=None):
    """Carry out cache_keep's moves and set length to n_keep."""
    c = cache
    budget = src.shape[-1]
    _call(c, "ab_cache_compact", c.struct, budget, _arr(src, torch.int32, (c.B, c.Hk, budget), c, "src"),
          _arr(n_keep, torch.int32, (c.B,), c, "n_keep"), _flag(dev_flag, c))
