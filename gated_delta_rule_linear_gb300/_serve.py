"""ctypes binding of the serving operators of libla.so: include/la_serve.h under
the same names, and wrappers that take torch CUDA tensors.

As in ``_layer``: argument marshalling only, on the device of the tensors, and a
non-zero status raises ``LAError``.
"""
from __future__ import annotations

import ctypes
import os

from ._binding import HEADER, _ptr
from . import _binding
from . import _layer
from ._layer import LAYER_CONSTANTS, _at, _check, _flag, _index, _launch, _rows

SERVE_HEADER = os.path.join(os.path.dirname(HEADER), "la_serve.h")

_P, _I, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
SERVE_SIGNATURES = {
    "la_cache_append": ([_P] * 11 + [_I] * 12 + [_L] * 5 + [_I, _P], _I),
    "la_paged_attn": ([_P] * 7 + [_I] * 7 + [_L] + [_I] * 2 + [_F] + [_L] * 2 + [_I, _P], _I),
    "la_beam_select": ([_P] * 6 + [_I] * 4 + [_L] + [_I] * 2 + [_P], _I),
    "la_beam_states": ([_P] * 3 + [_I] * 4 + [_L] * 3 + [_P], _I),
    "la_beam_cache": ([_P] * 5 + [_I] * 5 + [_L] + [_I] + [_L] * 3 + [_P], _I),
}


def _fn(name):
    f = _layer._fns.get(name)
    if f is None:
        f = getattr(_binding.load_library(), name)
        f.argtypes, f.restype = SERVE_SIGNATURES[name]
        _layer._fns[name] = f
    return f


def _run(name, *args):
    rc = (_layer._fns.get(name) or _fn(name))(*args)
    if rc != 0:
        raise _binding.LAError(rc, _binding.la_last_error())


# ---- raw C entry points (same names and argument order as la_serve.h) --------

def la_cache_append(q, k, v, q_out, k_cache, v_cache, table, lens, cu_seqlens, pos, freq, n_axes, s0, s1, s2, n_seq,
                    total, H, Hk, d, page_size, n_pages, max_pages, ld_table, ldq, ldk, ldv, ld_page, flags, stream):
    return _fn("la_cache_append")(_ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(table),
                                  _ptr(lens), _ptr(cu_seqlens), _ptr(pos), _ptr(freq), n_axes, s0, s1, s2, n_seq,
                                  total, H, Hk, d, page_size, n_pages, max_pages, ld_table, ldq, ldk, ldv, ld_page,
                                  flags, stream)


def la_paged_attn(q, k_cache, v_cache, o, lse, table, lens, n, H, Hk, d, page_size, n_pages, max_pages, ld_table,
                  max_len, window, scale, ldq, ld_page, flags, stream):
    return _fn("la_paged_attn")(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), _ptr(table), _ptr(lens), n,
                                H, Hk, d, page_size, n_pages, max_pages, ld_table, max_len, window, scale, ldq, ld_page,
                                flags, stream)


def la_beam_select(logits, scores, done, scores_out, parent, token, B, W, V, K, ld, eos, flags, stream):
    return _fn("la_beam_select")(_ptr(logits), _ptr(scores), _ptr(done), _ptr(scores_out), _ptr(parent), _ptr(token),
                                 B, W, V, K, ld, eos, flags, stream)


def la_beam_states(pool, slots, parent, B, W, n_slots, layers, row_bytes, ld_row, ld_layer, stream):
    return _fn("la_beam_states")(_ptr(pool), _ptr(slots), _ptr(parent), B, W, n_slots, layers, row_bytes, ld_row,
                                 ld_layer, stream)


def la_beam_cache(k_cache, v_cache, table, lens, parent, B, W, page_size, n_pages, max_pages, ld_table, layers,
                  token_bytes, ld_page, ld_layer, stream):
    return _fn("la_beam_cache")(_ptr(k_cache), _ptr(v_cache), _ptr(table), _ptr(lens), _ptr(parent), B, W, page_size,
                                n_pages, max_pages, ld_table, layers, token_bytes, ld_page, ld_layer, stream)


# ---- torch-tensor wrappers -----------------------------------------------------

def _inner(t, name, lead):
    """Strides of t's first ``lead`` dimensions; the others must be dense, and rows must not overlap."""
    shape, stride = t.shape, t.stride()
    n = 1
    for i in range(t.dim() - 1, -1, -1):
        if i >= lead:
            if shape[i] > 1 and stride[i] != n:
                raise ValueError(f"{name}: dimensions {lead} and up must be dense")
            n *= shape[i]
    at = n
    out = []
    for i in range(lead - 1, -1, -1):
        s = stride[i] if shape[i] > 1 else max(stride[i], at)
        if s < at:
            raise ValueError(f"{name}: dimension {i} overlaps itself or the next")
        out.append(s)
        at = s * max(shape[i], 1)
    return out[::-1]


def _caches(k_cache, v_cache, lead, idx, dtype):
    """Page (and layer) strides of the two pools, which must agree."""
    if k_cache.dim() != lead + 3 or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be one shape of {lead + 3} dimensions, got {tuple(k_cache.shape)}, "
                         f"{tuple(v_cache.shape)}")
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.get_device() != idx or not t.is_cuda:
            raise ValueError(f"{name} must be on CUDA device {idx}, got {t.device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if k_cache.is_contiguous() and v_cache.is_contiguous():
        return k_cache.stride()[:lead]
    ld = _inner(k_cache, "k_cache", lead)
    if _inner(v_cache, "v_cache", lead) != ld:
        raise ValueError("k_cache and v_cache must have the same strides")
    return ld


def _table(table, lens, n, idx):
    """(entries of a row, row stride) of a page table, with its lengths checked."""
    import torch
    if table.dim() != 2 or table.shape[0] != n or table.dtype is not torch.int32 or table.get_device() != idx:
        raise ValueError(f"table must be int32 [{n}, pages] on CUDA device {idx}")
    _check(lens, "lens", torch.int32, (n,), idx)
    width = table.shape[1]
    step, unit = table.stride()
    if (width > 1 and unit != 1) or (n > 1 and step < width):
        raise ValueError("table: the entries of a row must be dense, and rows apart")
    return width, step if n > 1 and step > width else width


def cache_append(q, k, v, k_cache, v_cache, table, lens, freq=None, pos=None, sections=None, interleaved=False,
                 cu_seqlens=None, q_out=None, stream=None):
    """New tokens into a paged cache, keys and queries turned on the way
    (la_cache_append). q [total,H,d] (or None), k, v [total,Hk,d], token stride
    free; k_cache, v_cache [pages,page_size,Hk,d], page stride free, changed in
    place; table int32 [n,max_pages]; lens int32 [n], the new tokens counted;
    cu_seqlens int32 [n+1] (None: one token for each sequence). freq float64
    [pairs], pos int32 [total,axes] (None: the place in the cache) and sections
    as rotary; freq None: no rotation. Returns the turned queries (or None)."""
    import torch
    idx, dt, i32 = _index(k, "k"), k.dtype, torch.int32
    ldk, ldv = _rows(k, "k"), _rows(v, "v")
    N, Hk, d = k.shape
    if v.shape != k.shape or v.dtype is not dt or v.get_device() != idx:
        raise ValueError("v must have k's shape, dtype and device")
    H = ldq = 0
    if q is not None:
        ldq = _rows(q, "q")
        Nq, H, dq = q.shape
        if Nq != N or dq != d or q.dtype is not dt or q.get_device() != idx:
            raise ValueError("q and k must agree in tokens, channels, dtype and device")
    n = N if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", i32, (n + 1,), idx)
    (ld_page,) = _caches(k_cache, v_cache, 1, idx, dt)
    if tuple(k_cache.shape[2:]) != (Hk, d):
        raise ValueError(f"caches must be [pages, page_size, {Hk}, {d}], got {tuple(k_cache.shape)}")
    width, ld_table = _table(table, lens, n, idx)
    axes, s = 0, (0, 0, 0)
    if freq is not None:
        pairs = freq.numel()
        s = (pairs,) if sections is None else tuple(sections)
        axes = len(s)
        if sum(s) != pairs or not 1 <= axes <= 3:
            raise ValueError("sections: the pairs of one to three axes, as many as freq has")
        s = (s + (0, 0))[:3]
    _check(freq, "freq", torch.float64, (s[0] + s[1] + s[2],), idx)
    _check(pos, "pos", i32, (N, axes), idx)
    _check(q_out, "q_out", dt, (N, H, d), idx)
    flags = _flag(dt) | (LAYER_CONSTANTS["LA_ROT_INTERLEAVED"] if interleaved else 0)

    def body(handle):
        a = None if q is None else q.new_empty((N, H, d)) if q_out is None else q_out
        _run("la_cache_append", _at(q), k.data_ptr(), v.data_ptr(), _at(a), k_cache.data_ptr(), v_cache.data_ptr(),
             table.data_ptr(), lens.data_ptr(), _at(cu_seqlens), _at(pos), _at(freq), axes, *s, n, N, H, Hk, d,
             k_cache.shape[1], k_cache.shape[0], width, ld_table, ldq, ldk, ldv, ld_page, flags, handle)
        return a

    return _launch(idx, stream, body)


def paged_attn(q, k_cache, v_cache, table, lens, scale=None, window=0, max_len=0, with_lse=False, o=None, stream=None):
    """Attention of one new token of each sequence over a paged cache
    (la_paged_attn). q [n,H,d] (bf16 or fp32, token stride free); k_cache,
    v_cache [pages,page_size,Hk,d], page stride free; table int32
    [n,max_pages]; lens int32 [n]; scale None: d^-1/2; window > 0: the last
    places only. Returns (o [n,H,d], lse fp32 [n,H] or None)."""
    import torch
    ldq = _rows(q, "q")
    idx, dt = _index(q, "q"), q.dtype
    n, H, d = q.shape
    (ld_page,) = _caches(k_cache, v_cache, 1, idx, dt)
    pages, size, Hk, dk = k_cache.shape
    if dk != d:
        raise ValueError(f"caches must have q's {d} channels, got {dk}")
    width, ld_table = _table(table, lens, n, idx)
    _check(o, "o", dt, (n, H, d), idx)
    flags = _flag(dt)

    def body(handle):
        out = q.new_empty((n, H, d)) if o is None else o
        lse = q.new_empty((n, H), dtype=torch.float32) if with_lse else None
        _run("la_paged_attn", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), _at(lse),
             table.data_ptr(), lens.data_ptr(), n, H, Hk, d, size, pages, width, ld_table, max_len, window,
             d ** -0.5 if scale is None else scale, ldq, ld_page, flags, handle)
        return out, lse

    return _launch(idx, stream, body)


def beam_select(logits, scores, K=None, done=None, eos=0, stream=None):
    """Beam search's step (la_beam_select). logits [B,W,V] (bf16 or fp32, row
    stride free); scores fp32 [B,W]; done bool or uint8 [B,W] or None; K None: W.
    Returns (scores fp32, parent int32, token int32), each [B,K], best first."""
    import torch
    if logits.dim() != 3:
        raise ValueError(f"logits must be [B, W, V], got {tuple(logits.shape)}")
    idx, f32, i32 = _index(logits, "logits"), torch.float32, torch.int32
    B, W, V = logits.shape
    sb, sw, sv = logits.stride()
    ld = V if logits.is_contiguous() else sw if W > 1 else sb if B > 1 else V
    if (V > 1 and sv != 1) or (W > 1 and B > 1 and sb != W * sw) or ld < V:
        raise ValueError("logits: a row must be dense, and rows at one stride")
    K = W if K is None else K
    _check(scores, "scores", f32, (B, W), idx)
    if done is not None:
        _check(done, "done", torch.bool if done.dtype is torch.bool else torch.uint8, (B, W), idx)
    flags = _flag(logits.dtype)

    def body(handle):
        best = scores.new_empty((B, K))
        parent, token = scores.new_empty((B, K), dtype=i32), scores.new_empty((B, K), dtype=i32)
        _run("la_beam_select", logits.data_ptr(), scores.data_ptr(), _at(done), best.data_ptr(), parent.data_ptr(),
             token.data_ptr(), B, W, V, K, ld, eos, flags, handle)
        return best, parent, token

    return _launch(idx, stream, body)


def beam_states(pool, parent, slots=None, layered=False, stream=None):
    """Rows of a pool of states after a beam step (la_beam_states), in place:
    row slots[b*W + w] becomes what row slots[b*W + parent[b,w]] was. pool
    [rows, ...], or [layers, rows, ...] with ``layered``, any dtype, a row dense;
    parent int32 [B,W]; slots int32 [B*W] (None: row b*W + w). Returns pool."""
    import torch
    idx, lead = _index(pool, "pool"), 2 if layered else 1
    if pool.dim() < lead:
        raise ValueError(f"pool must have {lead} dimensions or more, got {tuple(pool.shape)}")
    if parent.dim() != 2:
        raise ValueError(f"parent must be [B, W], got {tuple(parent.shape)}")
    B, W = parent.shape
    _check(parent, "parent", torch.int32, (B, W), idx)
    _check(slots, "slots", torch.int32, (B * W,), idx)
    e = pool.element_size()
    ld = _inner(pool, "pool", lead)
    row = 1
    for s in pool.shape[lead:]:
        row *= s

    def body(handle):
        _run("la_beam_states", pool.data_ptr(), _at(slots), parent.data_ptr(), B, W, pool.shape[lead - 1],
             pool.shape[0] if layered else 1, row * e, ld[-1] * e, ld[0] * e if layered else 0, handle)
        return pool

    return _launch(idx, stream, body)


def beam_cache(k_cache, v_cache, table, lens, parent, layered=False, stream=None):
    """A paged cache after a beam step (la_beam_cache), in place: full pages are
    shared with the parent by the table, the open page's tokens are copied.
    k_cache, v_cache [pages,page_size,Hk,d], or [layers,pages,page_size,Hk,d]
    with ``layered``, page and layer strides free; table int32 [B*W,max_pages];
    lens int32 [B*W]; parent int32 [B,W]. Returns (k_cache, v_cache, table)."""
    import torch
    idx, lead = _index(k_cache, "k_cache"), 2 if layered else 1
    if parent.dim() != 2:
        raise ValueError(f"parent must be [B, W], got {tuple(parent.shape)}")
    B, W = parent.shape
    _check(parent, "parent", torch.int32, (B, W), idx)
    ld = _caches(k_cache, v_cache, lead, idx, k_cache.dtype)
    width, ld_table = _table(table, lens, B * W, idx)
    pages, size, Hk, d = k_cache.shape[lead - 1:]
    e = k_cache.element_size()

    def body(handle):
        _run("la_beam_cache", k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
             parent.data_ptr(), B, W, size, pages, width, ld_table, k_cache.shape[0] if layered else 1, Hk * d * e,
             ld[-1] * e, ld[0] * e if layered else 0, handle)
        return k_cache, v_cache, table

    return _launch(idx, stream, body)
