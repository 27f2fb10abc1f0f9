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
# Calls of a few tokens are bound by their host side: the wrappers look at each tensor's attributes once, and leave
# the general case (and the reasons of a refusal) to functions of their own.

torch = None  # imported by the first call
_INT = range(-(1 << 31), 1 << 31)  # what an int argument holds: ctypes would pass the low 32 bits of others


def _setup():
    global torch, _FLAGS
    import torch as t
    _FLAGS = {t.bfloat16: 0, t.float32: _binding.CONSTANTS["LA_F32"]}
    torch = t
    return t


def _handle(idx, stream):
    """The current stream's handle where a call runs there, on the current device; else None."""
    return torch._C._cuda_getCurrentRawStream(idx) if stream is None and torch._C._cuda_getDevice() == idx else None


def _inner(t, name, lead):
    """Strides of t's first ``lead`` dimensions, one inside the other in any order; the others must be dense, and rows
    must not overlap."""
    shape, stride = t.shape, t.stride()
    n = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] > 1 and stride[i] != n:
            raise ValueError(f"{name}: dimensions {lead} and up must be dense")
        n *= max(shape[i], 1)  # (as torch's strides of empty tensors)
    out = [n] * lead
    end = n  # elements that the dimensions inside reach over
    for s, i in sorted((stride[i], i) for i in range(lead) if shape[i] > 1):
        if s < end:
            raise ValueError(f"{name}: rows of dimension {i} overlap")
        out[i] = s
        end += s * (shape[i] - 1)
    return tuple(out)


def _caches(k_cache, v_cache, lead, idx, dtype):
    """Shape and page (and layer) strides of the two pools, which must agree."""
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != lead + 3 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be one shape of {lead + 3} dimensions, got {tuple(shape)}, "
                         f"{tuple(v_cache.shape)}")
    if k_cache.get_device() != idx or v_cache.get_device() != idx:
        raise ValueError(f"k_cache and v_cache must be on CUDA device {idx}, got {k_cache.device}, {v_cache.device}")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        raise TypeError(f"k_cache and v_cache must be {dtype}, got {k_cache.dtype}, {v_cache.dtype}")
    if v_cache.stride() == stride and lead == 1:
        _, size, Hk, d = shape
        if stride[1:] == (Hk * d, d, 1) and stride[0] >= size * Hk * d:
            return shape, stride[:1]
    ld = _inner(k_cache, "k_cache", lead)
    if _inner(v_cache, "v_cache", lead) != ld:
        raise ValueError("k_cache and v_cache must have the same strides")
    return shape, ld


def _table(table, lens, n, idx):
    """(entries of a row, row stride) of a page table, with its lengths checked."""
    shape, i32 = table.shape, torch.int32
    if len(shape) != 2 or shape[0] != n or table.dtype is not i32 or table.get_device() != idx:
        raise ValueError(f"table must be int32 [{n}, pages] on CUDA device {idx}")
    if lens.dtype is not i32 or lens.shape != (n,) or lens.get_device() != idx or not lens.is_contiguous():
        _check(lens, "lens", i32, (n,), idx)
    width = shape[1]
    step, unit = table.stride()
    if unit == 1 and step >= width:
        return width, step if step > width else width
    if (width > 1 and unit != 1) or (n > 1 and step < width):
        raise ValueError("table: the entries of a row must be dense, and rows apart")
    return width, width if n <= 1 else step


def cache_append(q, k, v, k_cache, v_cache, table, lens, freq=None, pos=None, sections=None, interleaved=False,
                 cu_seqlens=None, q_out=None, stream=None):
    """New tokens into a paged cache, keys and queries turned on the way
    (la_cache_append). q [total,H,d] (or None), k, v [total,Hk,d], token stride
    free; k_cache, v_cache [pages,page_size,Hk,d], page stride free, changed in
    place; table int32 [n,max_pages]; lens int32 [n], the new tokens counted;
    cu_seqlens int32 [n+1] (None: one token for each sequence). freq float64
    [pairs], pos int32 [total,axes] (None: the place in the cache) and sections
    as rotary; freq None: no rotation. Returns the turned queries (or None)."""
    t = torch or _setup()
    idx, dt, shape, ldk, ldv = k.get_device(), k.dtype, k.shape, _rows(k, "k"), _rows(v, "v")
    if idx < 0:
        _index(k, "k")
    N, Hk, d = shape
    if v.shape != shape or v.dtype is not dt or v.get_device() != idx:
        raise ValueError("v must have k's shape, dtype and device")
    H = ldq = 0
    if q is not None:
        ldq = _rows(q, "q")
        Nq, H, dq = q.shape
        if Nq != N or dq != d or q.dtype is not dt or q.get_device() != idx:
            raise ValueError("q and k must agree in tokens, channels, dtype and device")
    n = N
    if cu_seqlens is not None:
        n = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", t.int32, (n + 1,), idx)
    pages, (ld_page,) = _caches(k_cache, v_cache, 1, idx, dt)
    if pages[2] != Hk or pages[3] != d:
        raise ValueError(f"caches must be [pages, page_size, {Hk}, {d}], got {tuple(pages)}")
    width, ld_table = _table(table, lens, n, idx)
    axes, s0, s1, s2 = 0, 0, 0, 0
    if freq is not None:
        s0 = pairs = freq.numel()
        axes = 1
        if sections is not None:
            axes = len(sections)
            if sum(sections) != pairs or not 1 <= axes <= 3:
                raise ValueError("sections: the pairs of one to three axes, as many as freq has")
            s0, s1, s2 = (*sections, 0, 0)[:3]
        _check(freq, "freq", t.float64, (pairs,), idx)
    if pos is not None:
        _check(pos, "pos", t.int32, (N, axes), idx)
    if q_out is not None:
        _check(q_out, "q_out", dt, (N, H, d), idx)
    flags = _FLAGS.get(dt)
    if flags is None:
        _flag(dt)
    if interleaved:
        flags |= LAYER_CONSTANTS["LA_ROT_INTERLEAVED"]

    def body(handle):
        a = None if q is None else q_out
        if a is None and q is not None:
            a = t.empty((N, H, d), dtype=dt, device=q.device)
        _run("la_cache_append", None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
             None if a is None else a.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(),
             lens.data_ptr(), _at(cu_seqlens), _at(pos), _at(freq), axes, s0, s1, s2, n, N, H, Hk, d, pages[1], pages[0],
             width, ld_table, ldq, ldk, ldv, ld_page, flags, handle)
        return a

    handle = _handle(idx, stream)
    return body(handle) if handle is not None else _launch(idx, stream, body)


def paged_attn(q, k_cache, v_cache, table, lens, scale=None, window=0, max_len=0, with_lse=False, o=None, stream=None):
    """Attention of one new token of each sequence over a paged cache
    (la_paged_attn). q [n,H,d] (bf16 or fp32, token stride free); k_cache,
    v_cache [pages,page_size,Hk,d], page stride free; table int32
    [n,max_pages]; lens int32 [n]; scale None: d^-1/2; window > 0: the last
    places only. Returns (o [n,H,d], lse fp32 [n,H] or None)."""
    t = torch or _setup()
    idx, dt, ldq = q.get_device(), q.dtype, _rows(q, "q")
    if idx < 0:
        _index(q, "q")
    n, H, d = q.shape
    pages, (ld_page,) = _caches(k_cache, v_cache, 1, idx, dt)
    if pages[3] != d:
        raise ValueError(f"caches must have q's {d} channels, got {pages[3]}")
    width, ld_table = _table(table, lens, n, idx)
    if max_len not in _INT or window not in _INT:
        raise ValueError(f"max_len and window must be below 2^31, got {max_len}, {window}")
    if o is not None:
        _check(o, "o", dt, (n, H, d), idx)
    flags = _FLAGS.get(dt)
    if flags is None:
        _flag(dt)

    def body(handle):
        out = t.empty((n, H, d), dtype=dt, device=q.device) if o is None else o
        lse = t.empty((n, H), dtype=t.float32, device=q.device) if with_lse else None
        _run("la_paged_attn", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), _at(lse),
             table.data_ptr(), lens.data_ptr(), n, H, pages[2], d, pages[1], pages[0], width, ld_table, max_len, window,
             d ** -0.5 if scale is None else scale, ldq, ld_page, flags, handle)
        return out, lse

    handle = _handle(idx, stream)
    return body(handle) if handle is not None else _launch(idx, stream, body)


def beam_select(logits, scores, K=None, done=None, eos=0, stream=None):
    """Beam search's step (la_beam_select). logits [B,W,V] (bf16 or fp32, row
    stride free); scores fp32 [B,W]; done bool or uint8 [B,W] or None; K None: W.
    Returns (scores fp32, parent int32, token int32), each [B,K], best first."""
    t = torch or _setup()
    shape, idx, f32, i32 = logits.shape, logits.get_device(), t.float32, t.int32
    if len(shape) != 3:
        raise ValueError(f"logits must be [B, W, V], got {tuple(shape)}")
    if idx < 0:
        _index(logits, "logits")
    B, W, V = shape
    sb, sw, sv = logits.stride()
    if sv == 1 and sb == W * sw and sw >= V:
        ld = sw
    else:
        ld = V if logits.is_contiguous() else sw if W > 1 else sb if B > 1 else V
        if (V > 1 and sv != 1) or (W > 1 and B > 1 and sb != W * sw) or ld < V:
            raise ValueError("logits: a row must be dense, and rows at one stride")
    K = W if K is None else K
    if K not in _INT or eos not in _INT:
        raise ValueError(f"K and eos must be below 2^31, got {K}, {eos}")
    _check(scores, "scores", f32, (B, W), idx)
    if done is not None:
        _check(done, "done", t.bool if done.dtype is t.bool else t.uint8, (B, W), idx)
    flags = _FLAGS.get(logits.dtype)
    if flags is None:
        _flag(logits.dtype)

    def body(handle):
        if K == W:
            best = t.empty_like(scores)
        else:
            best = t.empty((B, K), dtype=f32, device=scores.device)
        parent, token = t.empty_like(best, dtype=i32), t.empty_like(best, dtype=i32)
        _run("la_beam_select", logits.data_ptr(), scores.data_ptr(), _at(done), best.data_ptr(), parent.data_ptr(),
             token.data_ptr(), B, W, V, K, ld, eos, flags, handle)
        return best, parent, token

    handle = _handle(idx, stream)
    return body(handle) if handle is not None else _launch(idx, stream, body)


def beam_states(pool, parent, slots=None, layered=False, stream=None):
    """Rows of a pool of states after a beam step (la_beam_states), in place:
    row slots[b*W + w] becomes what row slots[b*W + parent[b,w]] was. pool
    [rows, ...], or [layers, rows, ...] with ``layered``, any dtype, a row dense;
    parent int32 [B,W]; slots int32 [B*W] (None: row b*W + w). Returns pool."""
    if torch is None:
        _setup()
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

    handle = _handle(idx, stream)
    return body(handle) if handle is not None else _launch(idx, stream, body)


def beam_cache(k_cache, v_cache, table, lens, parent, layered=False, stream=None):
    """A paged cache after a beam step (la_beam_cache), in place: full pages are
    shared with the parent by the table, the open page's tokens are copied.
    k_cache, v_cache [pages,page_size,Hk,d], or [layers,pages,page_size,Hk,d]
    with ``layered``, page and layer strides free; table int32 [B*W,max_pages];
    lens int32 [B*W]; parent int32 [B,W]. Returns (k_cache, v_cache, table)."""
    if torch is None:
        _setup()
    idx, lead = _index(k_cache, "k_cache"), 2 if layered else 1
    if parent.dim() != 2:
        raise ValueError(f"parent must be [B, W], got {tuple(parent.shape)}")
    B, W = parent.shape
    _check(parent, "parent", torch.int32, (B, W), idx)
    shape, ld = _caches(k_cache, v_cache, lead, idx, k_cache.dtype)
    width, ld_table = _table(table, lens, B * W, idx)
    pages, size, Hk, d = shape[lead - 1:]
    e = k_cache.element_size()

    def body(handle):
        _run("la_beam_cache", k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
             parent.data_ptr(), B, W, size, pages, width, ld_table, k_cache.shape[0] if layered else 1, Hk * d * e,
             ld[-1] * e, ld[0] * e if layered else 0, handle)
        return k_cache, v_cache, table

    handle = _handle(idx, stream)
    return body(handle) if handle is not None else _launch(idx, stream, body)
