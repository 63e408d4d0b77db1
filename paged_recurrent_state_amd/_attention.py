"""ctypes binding of the attention layers' entry points (include/gdn_attention.h):
rotary positions, norms before them, the append to a paged key/value cache (of the rows' type or of
8 bits) and the read back, and attention over it.

Argument marshalling only, as in ``_lib``: every step runs in the HIP library on
the tensors' device, on torch's current stream, and there is no fallback.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from ._lib import (GDN_INDEX_INT32, GDN_INDEX_INT64, _AttentionC, _CacheC, _need, _NormC, _RopeC, _RowsC, _run, _ScalesC,
                   _ScalingC, _workspace, load)
from ._lib import _stream as _stream_of_device

# element types (GDN_TYPE_*)
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
E4M3 = torch.float8_e4m3fn  # element type of a cache of 8 bits
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


def _stream(dev: torch.device):
    """torch's current stream on ``dev``: its handle alone, since at small sizes a
    ``torch.cuda.Stream`` object would cost as much as the kernel."""
    if dev.type != "cuda" or dev.index is None:
        return _stream_of_device(dev)
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _no_tangents(call: str, *tensors):
    """Refuses dual tensors (those of forward-mode differentiation), whose tangents the kernels do not see."""
    if any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError(f"{call} has no forward-mode derivative: its inputs must not be dual tensors")


def _dense(shape, dtype, dev):
    """A new dense [tokens, heads, dim] tensor and its gdn_rows_t."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    return t, _RowsC(t.data_ptr(), shape[1] * shape[2], shape[2])


def _dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _rows(t, name: str, dtype, dev, heads: Optional[int] = None, tokens: Optional[int] = None,
          dim: Optional[int] = None) -> _RowsC:
    """[tokens, heads, dim] with a dense last dimension, as gdn_rows_t."""
    _need(t, name, dtype, dev, contiguous=False)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(t.shape)}")
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) or (dim is not None and d != dim):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}], got {tuple(t.shape)}")
    ts, hs, ds = t.stride()
    if ds != 1 and d > 1:
        raise ValueError(f"the last dimension of {name} must be dense")
    return _RowsC(t.data_ptr(), ts, hs)


def _cache(k_cache, v_cache, page_indices, page_indptr, page_size, last_page_len, dtype, dev, dim) -> _CacheC:
    """[pages, page_size, kv heads, dim] keys and values of equal strides, and their page table."""
    _need(k_cache, "k_cache", dtype, dev, contiguous=False)
    _need(v_cache, "v_cache", dtype, dev, contiguous=False)
    if k_cache.dim() != 4 or k_cache.shape[1] != page_size or k_cache.shape[3] != dim:
        raise ValueError(f"k_cache must be [pages, {page_size}, kv heads, {dim}], got {tuple(k_cache.shape)}")
    if v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache must have the shape of k_cache, got {tuple(v_cache.shape)}")
    stride = k_cache.stride()
    # (a dimension of one has no step, whatever its stride says)
    if v_cache.stride() != stride and any(a != b and n > 1 for a, b, n in zip(stride, v_cache.stride(), k_cache.shape)):
        raise ValueError("k_cache and v_cache must have the same strides")
    if stride[3] != 1 and dim > 1:
        raise ValueError("the last dimension of the caches must be dense")
    _need(page_indices, "page_indices", torch.int32, dev)
    _need(page_indptr, "page_indptr", torch.int32, dev)
    _need(last_page_len, "last_page_len", torch.int32, dev)
    B = last_page_len.shape[0]
    if page_indptr.shape[0] != B + 1:
        raise ValueError("page_indptr must have one entry more than last_page_len")
    # an empty tensor has no storage: a stand-in that is never read
    idx = page_indices if page_indices.numel() else page_indptr
    k, v = (c if c.numel() else page_indptr for c in (k_cache, v_cache))
    return _CacheC(k.data_ptr(), v.data_ptr(), stride[0] if k_cache.shape[0] > 1 else 0, stride[1], stride[2], page_size, B,
                   idx.data_ptr(), page_indptr.data_ptr(), last_page_len.data_ptr())


def _scales(k_scale, v_scale, k_cache, page_size: int, dev) -> _ScalesC:
    """[pages, blocks, kv heads] scales of an 8-bit cache's keys and values, of equal strides."""
    if k_scale is None or v_scale is None:
        raise ValueError("an 8-bit cache needs k_scale and v_scale, and no other takes them")
    _need(k_scale, "k_scale", torch.float32, dev, contiguous=False)
    _need(v_scale, "v_scale", torch.float32, dev, contiguous=False)
    shape, (pages, _, heads, _) = k_scale.shape, k_cache.shape
    if len(shape) != 3 or shape[0] != pages or shape[2] != heads or not shape[1]:
        raise ValueError(f"k_scale must be [{pages}, blocks of a page, {heads}], got {tuple(shape)}")
    if v_scale.shape != shape:
        raise ValueError(f"v_scale must have the shape of k_scale, got {tuple(v_scale.shape)}")
    stride = k_scale.stride()
    if v_scale.stride() != stride and any(a != b and n > 1 for a, b, n in zip(stride, v_scale.stride(), shape)):
        raise ValueError("k_scale and v_scale must have the same strides")
    blocks = shape[1]
    if page_size % blocks:
        raise ValueError(f"pages of {page_size} tokens do not divide into {blocks} blocks")
    # (no pages: stand-ins that are never read)
    k, v = (x.data_ptr() if x.numel() else 4 for x in (k_scale, v_scale))
    return _ScalesC(k, v, *stride, page_size // blocks)


def _norm(q_weight, k_weight, eps: float, offset: float, dtype, dim: int, dev) -> _NormC:
    """Weights [dim] of one type, the rows' or fp32; None: not normed."""
    # (as few questions as there can be: at one token the host's time is all there is)
    first = q_weight if q_weight is not None else k_weight
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor):
            raise TypeError("the norm's weights must be tensors")
        if w.dtype != first.dtype or (w.dtype != dtype and w.dtype != torch.float32):
            raise TypeError(f"the norm's weights must be of one type, {dtype} or torch.float32, got {w.dtype}")
        if w.device != dev:
            raise ValueError(f"the norm's weights are on {w.device}, expected {dev}")
        if w.shape != (dim,) or not w.is_contiguous():
            raise ValueError(f"the norm's weights must be contiguous [{dim}], got {tuple(w.shape)}")
    return _NormC(None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
                  DTYPES[dtype if first is None else first.dtype], float(eps), float(offset))


def _rope(table, interleaved: bool, transposed: bool, dev) -> _RopeC:
    _need(table, "table", torch.float32, dev)
    if table.dim() != 2:
        raise ValueError(f"table must be [positions, rot_dim], got {tuple(table.shape)}")
    return _RopeC(table.data_ptr(), table.shape[0], table.shape[1], bool(interleaved), transposed)


def _cu(cu_seqlens, B: int, dev):
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if cu_seqlens.shape[0] != B + 1:
        raise ValueError("cu_seqlens must have one entry more than last_page_len")
    return cu_seqlens.data_ptr()


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "plain",
               factor: float = 1.0, original: float = 0.0, low_turns: float = 1.0,
               high_turns: float = 4.0, magnitude: float = 1.0, device="cuda") -> torch.Tensor:
    """[positions, rot_dim] fp32: cosines, then sines, of ``position * f_i``, computed in fp64.

    ``f_i = base^(-2 i / rot_dim)``, for longer contexts changed by ``scaling``:
    "linear" (``f_i / factor``), "base" (``base * factor^(rot_dim / (rot_dim - 2))``) or "bands"
    (pairs that turn ``low_turns`` times or less over ``original`` tokens are slowed by
    ``factor``, those that turn ``high_turns`` times or more are kept, a linear blend
    between).  ``magnitude`` multiplies both."""
    lib = load()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    dev = torch.device(device)
    stream = _stream(dev)
    sc = _ScalingC(ROPE_SCALINGS[scaling], base, factor, original, low_turns, high_turns, magnitude)
    table = torch.empty(max(int(positions), 0), max(int(rot_dim), 0), dtype=torch.float32, device=dev)
    _run(dev, lib.gdn_rope_table, sc, table.data_ptr(), int(positions), int(rot_dim), stream)
    return table


def rope(q, k, table, positions, interleaved: bool = False, transposed: bool = False,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotate q [T, Hq, D] and k [T, Hk, D] (or None) at ``positions`` [T] (int32 or int64);
    returns (q_out, k_out), new dense tensors unless given (they may be q and k).

    ``table`` [positions, rot_dim] from ``rope_table``: the first ``rot_dim`` values of a head turn
    in pairs (i, i + rot_dim/2), or (2i, 2i + 1) with ``interleaved``.  ``transposed`` applies the
    transposed map.  A position outside the table gives NaN.

    q and k that require a gradient get it (the opposite map of the outputs' gradients); they and
    ``q_out`` or ``k_out`` exclude each other, and the table has no gradient.  There is no forward-mode
    derivative (dual tensors are refused)."""
    # (asked first and without a call: at one token the host's time is all there is)
    if forward_ad._current_level >= 0:
        _no_tangents("rope", q, k, table, q_out, k_out)
    if torch.is_grad_enabled() and (
            getattr(q, "requires_grad", False) or getattr(k, "requires_grad", False)
            or getattr(table, "requires_grad", False) or getattr(q_out, "requires_grad", False)
            or getattr(k_out, "requires_grad", False)):
        if table.requires_grad:
            raise RuntimeError("rope: the table has no gradient")
        if q_out is not None or k_out is not None:
            raise RuntimeError("rope: q_out and k_out take no part in automatic differentiation")
        return _Rope.apply(q, k, table, positions, interleaved, transposed)
    return _rope_rows(q, k, table, positions, interleaved, transposed, q_out, k_out)


class _Rope(torch.autograd.Function):
    """``rope`` and its gradient, which is linear: the opposite map of the outputs' gradients."""

    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved, transposed):
        ctx.save_for_backward(table, positions)
        ctx.map = interleaved, transposed
        ctx.set_materialize_grads(False)
        return _rope_rows(q, k, table, positions, interleaved, transposed, None, None)

    @staticmethod
    def backward(ctx, dq, dk):
        table, positions = ctx.saved_tensors
        interleaved, transposed = ctx.map
        # (a gradient that was broadcast, as a sum's, is laid out first)
        rows = [g if g is None or g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous() for g in (dq, dk)]
        given = [g for g in rows if g is not None]
        turned = iter(())
        if given:
            turned = iter(rope(given[0], given[1] if len(given) > 1 else None, table, positions, interleaved,
                               not transposed))
        dq, dk = (None if g is None else next(turned) for g in rows)
        return dq, dk, None, None, None, None


def _rope_rows(q, k, table, positions, interleaved, transposed, q_out, k_out, norm=None):
    lib = load()
    code, dev = _dtype(q, "q"), q.device
    stream = _stream(dev)
    T, Hq, D = q.shape if q.dim() == 3 else (None, None, None)
    qr = _rows(q, "q", q.dtype, dev)
    rp = _rope(table, interleaved, transposed, dev)
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 tensor")
    _need(positions, "positions", positions.dtype, dev)
    if tuple(positions.shape) != (T,):
        raise ValueError(f"positions must be [{T}], got {tuple(positions.shape)}")
    if q_out is None:
        q_out, qo = _dense((T, Hq, D), q.dtype, dev)
    else:
        qo = _rows(q_out, "q_out", q.dtype, dev, Hq, T, D)
    kr = ko = None
    Hk = 0
    if k is not None:
        kr = _rows(k, "k", q.dtype, dev, None, T, D)
        Hk = k.shape[1]
        if k_out is None:
            k_out, ko = _dense((T, Hk, D), q.dtype, dev)
        else:
            ko = _rows(k_out, "k_out", q.dtype, dev, Hk, T, D)
    tail = (rp, code, D, Hq, Hk, T, positions.data_ptr(),
            GDN_INDEX_INT64 if positions.dtype == torch.int64 else GDN_INDEX_INT32, qr, kr, qo, ko, stream)
    if norm is None:
        _run(dev, lib.gdn_rope, *tail)
    else:
        q_weight, k_weight, eps, offset = norm
        if q_weight is None or (k is not None and k_weight is None):
            raise ValueError("norm_rope needs the weights of the heads that it norms")
        nm = _norm(q_weight, None if k is None else k_weight, eps, offset, q.dtype, D, dev)
        _run(dev, lib.gdn_norm_rope, nm, *tail)
    return q_out, k_out


def rope_backward(dq, dk, table, positions, interleaved: bool = False,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of ``rope``'s inputs from those of its outputs (the transposed map)."""
    return rope(dq, dk, table, positions, interleaved, True, q_out, k_out)


def norm_rope(q, k, q_weight, k_weight, table, positions, eps: float = 1e-6, weight_offset: float = 0.0,
              interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``rope`` of the normed heads of q [T, Hq, D] and k [T, Hk, D] (or None), in one pass: each row x
    becomes ``x * rsqrt(mean(x^2) + eps) * (weight_offset + weight)`` before it turns.

    ``q_weight`` and ``k_weight`` [D] are of the rows' type or fp32, both alike (D at most 512).  q, k and
    the weights that require a gradient get it; ``q_out`` or ``k_out`` (they may be q and k) exclude
    that, and the table has no gradient.  There is no forward-mode derivative (dual tensors are refused)."""
    if forward_ad._current_level >= 0:
        _no_tangents("norm_rope", q, k, q_weight, k_weight, table, q_out, k_out)
    if torch.is_grad_enabled() and (
            getattr(q, "requires_grad", False) or getattr(k, "requires_grad", False)
            or getattr(q_weight, "requires_grad", False) or getattr(k_weight, "requires_grad", False)
            or getattr(table, "requires_grad", False) or getattr(q_out, "requires_grad", False)
            or getattr(k_out, "requires_grad", False)):
        if getattr(table, "requires_grad", False):
            raise RuntimeError("norm_rope: the table has no gradient")
        if q_out is not None or k_out is not None:
            raise RuntimeError("norm_rope: q_out and k_out take no part in automatic differentiation")
        return _NormRope.apply(q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved)
    return _rope_rows(q, k, table, positions, interleaved, False, q_out, k_out, (q_weight, k_weight, eps, weight_offset))


class _NormRope(torch.autograd.Function):
    """``norm_rope`` and ``norm_rope_backward``."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.more = eps, weight_offset, interleaved
        ctx.set_materialize_grads(False)
        return _rope_rows(q, k, table, positions, interleaved, False, None, None, (q_weight, k_weight, eps, weight_offset))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        # (a gradient that was broadcast, as a sum's, is laid out first)
        dq, dk = (g if g is None or g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous() for g in (dq, dk))
        rest = (table, positions, *ctx.more)
        none = (None,) * 5
        if dq is not None:
            keys = (None, None) if dk is None else (k, k_weight)
            dq, dk, dqw, dkw = norm_rope_backward(dq, dk, q, keys[0], q_weight, keys[1], *rest)
            return (dq, dk, dqw, dkw, *none)
        if dk is None:
            return (None,) * 9
        dk, _, dkw, _ = norm_rope_backward(dk, None, k, None, k_weight, None, *rest)
        return (None, dk, None, dkw, *none)


@lru_cache(maxsize=256)
def _backward_size(head_dim: int, num_q_heads: int, num_k_heads: int, tokens: int, device: int) -> int:
    return int(load().gdn_norm_rope_backward_workspace_size(head_dim, num_q_heads, num_k_heads, tokens))


def norm_rope_backward(dq, dk, q, k, q_weight, k_weight, table, positions, eps: float = 1e-6,
                       weight_offset: float = 0.0, interleaved: bool = False,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients (of q, of k, of q_weight, of k_weight) from those of ``norm_rope``'s outputs, dq
    [T, Hq, D] and dk [T, Hk, D], and its inputs; dk, k and k_weight may be None together.  The weights'
    gradients are sums over all rows, in an order that depends on the sizes alone."""
    if forward_ad._current_level >= 0:
        _no_tangents("norm_rope_backward", dq, dk, q, k, q_weight, k_weight, table)
    lib = load()
    code, dev = _dtype(q, "q"), q.device
    stream = _stream(dev)
    qr = _rows(q, "q", q.dtype, dev)
    T, Hq, D = q.shape
    gq = _rows(dq, "dq", q.dtype, dev, Hq, T, D)
    if (k is None) != (dk is None) or (k is None) != (k_weight is None) or q_weight is None:
        raise ValueError("norm_rope_backward takes dk, k and k_weight together, and q_weight")
    rp = _rope(table, interleaved, False, dev)
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 tensor")
    _need(positions, "positions", positions.dtype, dev)
    if tuple(positions.shape) != (T,):
        raise ValueError(f"positions must be [{T}], got {tuple(positions.shape)}")
    nm = _norm(q_weight, k_weight, eps, weight_offset, q.dtype, D, dev)
    q_grad, qo = _dense((T, Hq, D), q.dtype, dev)
    qw_grad = torch.empty_like(q_weight)
    k_grad = kw_grad = kr = gk = ko = kw = None
    Hk = 0
    if k is not None:
        kr = _rows(k, "k", q.dtype, dev, None, T, D)
        Hk = k.shape[1]
        gk = _rows(dk, "dk", q.dtype, dev, Hk, T, D)
        k_grad, ko = _dense((T, Hk, D), q.dtype, dev)
        kw_grad = torch.empty_like(k_weight)
        kw = kw_grad.data_ptr()
    ws = _workspace(workspace, _backward_size(D, Hq, Hk, T, dev.index), dev)
    if Hq == 0:
        qw_grad.zero_()
    if k is not None and Hk == 0:
        kw_grad.zero_()
    _run(dev, lib.gdn_norm_rope_backward, nm, rp, code, D, Hq, Hk, T, positions.data_ptr(),
         GDN_INDEX_INT64 if positions.dtype == torch.int64 else GDN_INDEX_INT32, qr, kr, gq, gk, qo, ko,
         qw_grad.data_ptr(), kw, ws.data_ptr(), ws.numel() * ws.element_size(), stream)
    return q_grad, k_grad, qw_grad, kw_grad


def kv_append_paged(k, v, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size: int,
                    last_page_len, table: Optional[torch.Tensor] = None, interleaved: bool = False,
                    q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, norm_offset: float = 0.0, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Write the new tokens' k and v [T, Hkv, D] to the paged caches [pages, page_size, Hkv, D]
    (any strides, the last dimension dense), in one launch (no gradient: a serving call, as the
    attention calls on these caches).

    ``table`` (``rope_table``) rotates the keys on the way, and ``q`` [T, Hq, D], when given, into
    ``q_out`` (returned; a new tensor unless given).  The page table is the one after the
    append; ``cu_seqlens`` [B + 1] gives each sequence's new tokens, None one token each.

    ``q_norm`` and ``k_norm`` [D] norm the queries and the keys before they turn, as ``norm_rope`` does
    (None: they pass).  Caches of 8 bits (``torch.float8_e4m3fn``, D 64, 128 or 256, rows of 16-bit
    types) take ``k_scale`` and ``v_scale`` [pages, page_size / block, Hkv] fp32, written with them: a power of
    two for each ``block`` tokens of a page and head (a multiple of 16), with which the block's largest
    value is at most 448.  A block that tokens are added to keeps its scale or takes the larger new one,
    its codes rounded to it; one that they open takes a new one.  With norms or scales, rows of ``q_out``
    behind ``cu_seqlens[-1]`` are left as they are."""
    lib = load()
    code, dev = _dtype(k, "k"), k.device
    stream = _stream(dev)
    kr = _rows(k, "k", k.dtype, dev)
    T, Hk, D = k.shape
    vr = _rows(v, "v", k.dtype, dev, Hk, T, D)
    coded = getattr(k_cache, "dtype", None) == E4M3
    cache = _cache(k_cache, v_cache, page_indices, page_indptr, int(page_size), last_page_len,
                   E4M3 if coded else k.dtype, dev, D)
    if k_cache.shape[2] != Hk:
        raise ValueError(f"the caches must have the {Hk} heads of k, got {k_cache.shape[2]}")
    cu = None if cu_seqlens is None else _cu(cu_seqlens, cache.num_seqs, dev)
    rp = None if table is None else _rope(table, interleaved, False, dev)
    qr = qo = None
    Hq = 0
    if q is not None:
        qr = _rows(q, "q", k.dtype, dev, None, T, D)
        Hq = q.shape[1]
        if q_out is None:
            q_out, qo = _dense((T, Hq, D), k.dtype, dev)
        else:
            qo = _rows(q_out, "q_out", k.dtype, dev, Hq, T, D)
    if q_norm is None and k_norm is None and not coded and k_scale is None and v_scale is None:
        _run(dev, lib.gdn_kv_append_paged, rp, code, D, Hq, Hk, cu, T, kr, vr, cache, qr, qo, stream)
        return q_out
    if q_norm is not None and q is None:
        raise ValueError("q_norm norms the queries: q is missing")
    if not coded and (k_scale is not None or v_scale is not None):
        raise ValueError(f"k_scale and v_scale belong to caches of {E4M3}")
    nm = None if q_norm is None and k_norm is None else _norm(q_norm, k_norm, eps, norm_offset, k.dtype, D, dev)
    sc = _scales(k_scale, v_scale, k_cache, int(page_size), dev) if coded else None
    _run(dev, lib.gdn_kv_append_paged_ext, nm, rp, code, D, Hq, Hk, cu, T, kr, vr, cache, sc, qr, qo, stream)
    return q_out


def kv_read_paged(cu_seqlens, total_tokens: int, k_cache, v_cache, page_indices, page_indptr, page_size: int,
                  last_page_len, k_scale, v_scale, dtype: torch.dtype = torch.bfloat16,
                  k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values [total_tokens, Hkv, D] of ``dtype`` (bf16, fp16 or fp32) back from caches of 8 bits,
    into new tensors unless given: rows ``cu_seqlens[b] ..`` (None: one row per sequence) hold the last so
    many tokens of sequence b, as ``kv_append_paged`` counts its new ones.  Rows whose sequence holds
    fewer are zeros; rows behind ``cu_seqlens[-1]`` are left as they are."""
    lib = load()
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, kv heads, dim]")
    dev = k_cache.device
    stream = _stream(dev)
    T, Hk, D = int(total_tokens), k_cache.shape[2], k_cache.shape[3]
    cache = _cache(k_cache, v_cache, page_indices, page_indptr, int(page_size), last_page_len, E4M3, dev, D)
    sc = _scales(k_scale, v_scale, k_cache, int(page_size), dev)
    cu = None if cu_seqlens is None else _cu(cu_seqlens, cache.num_seqs, dev)
    rows = []
    for name, out in (("k_out", k_out), ("v_out", v_out)):
        rows.append(_dense((max(T, 0), Hk, D), dtype, dev) if out is None
                    else (out, _rows(out, name, dtype, dev, Hk, T, D)))
    (k, kr), (v, vr) = rows
    _run(dev, lib.gdn_kv_read_paged, DTYPES[dtype], D, Hk, cu, T, cache, sc, kr, vr, stream)
    return k, v


@lru_cache(maxsize=256)
def _workspace_size(total_tokens: int, num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                    device: int, coded: bool) -> int:
    d = _AttentionC(num_q_heads, num_kv_heads, head_dim, 0, 0.0, 0.0, 0, 1)
    return int(load().gdn_attention_workspace_size_ext(d, coded, total_tokens, num_seqs))


def attention_workspace_size(total_tokens: int, num_seqs: int, num_q_heads: int, num_kv_heads: int,
                             head_dim: int, cache_dtype: Optional[torch.dtype] = None) -> int:
    """Bytes either attention call needs for at most that many query rows and sequences, over caches of any
    type, or of ``cache_dtype`` alone (those of 8 bits need less for up to 7 q-heads on a kv-head, and more beyond)."""
    d = _AttentionC(num_q_heads, num_kv_heads, head_dim, 0, 0.0, 0.0, 0, 1)
    if cache_dtype is None:
        return int(load().gdn_attention_workspace_size(d, int(total_tokens), int(num_seqs)))
    if cache_dtype not in (torch.bfloat16, torch.float16, E4M3):
        raise TypeError(f"cache_dtype must be bfloat16, float16 or {E4M3}, got {cache_dtype}")
    return int(load().gdn_attention_workspace_size_ext(d, cache_dtype == E4M3, int(total_tokens), int(num_seqs)))


def _attention(fn, q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size, last_page_len,
               scale, softcap, window, causal, return_lse, out, workspace, sinks, k_scale, v_scale):
    lib = load()
    code, dev = _dtype(q, "q"), q.device
    stream = _stream(dev)
    qr = _rows(q, "q", q.dtype, dev)
    T, Hq, D = q.shape
    coded = getattr(k_cache, "dtype", None) == E4M3
    cache = _cache(k_cache, v_cache, page_indices, page_indptr, int(page_size), last_page_len,
                   E4M3 if coded else q.dtype, dev, D)
    if not coded and (k_scale is not None or v_scale is not None):
        raise ValueError(f"k_scale and v_scale belong to caches of {E4M3}")
    # (the library takes what is not positive for its defaults)
    scale, softcap = 0.0 if scale is None else float(scale), 0.0 if softcap is None else float(softcap)
    if scale < 0.0 or softcap < 0.0:
        raise ValueError(f"scale and softcap must not be negative, got {scale} and {softcap}")
    window = int(window)
    if window >> 31:  # (the argument's 32 bits: no sequence is longer, and a negative one is refused)
        window = -1 if window < 0 else (1 << 31) - 1
    d = _AttentionC(Hq, k_cache.shape[2], D, code, scale, softcap, window, bool(causal))
    if out is None:
        out, o = _dense((T, Hq, D), q.dtype, dev)
    else:
        o = _rows(out, "out", q.dtype, dev, Hq, T, D)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if return_lse else None
    ws = _workspace(workspace, _workspace_size(T, cache.num_seqs, Hq, k_cache.shape[2], D, dev.index, coded), dev)
    tail = (o, lse.data_ptr() if return_lse else None, ws.data_ptr(), ws.numel() * ws.element_size(),
            stream)
    if fn == "prefill":
        head = (qr, _cu(cu_seqlens, cache.num_seqs, dev), T)
        plain, ext = lib.gdn_attention_prefill_paged, lib.gdn_attention_prefill_paged_ext
    else:
        if T != cache.num_seqs:
            raise ValueError(f"q must have one row per sequence ({cache.num_seqs}), got {T}")
        head, plain, ext = (qr,), lib.gdn_attention_decode_paged, lib.gdn_attention_decode_paged_ext
    if not coded and not sinks:
        _run(dev, plain, d, *head, cache, *tail)
    else:
        sinks = max(-1, min(int(sinks), (1 << 31) - 1))  # (the argument's 32 bits: the call refuses what is past its range)
        sc = _scales(k_scale, v_scale, k_cache, int(page_size), dev) if coded else None
        _run(dev, ext, d, sinks, *head, cache, sc, *tail)
    return (out, lse) if return_lse else out


def attention_prefill_paged(q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size: int,
                            last_page_len, scale: Optional[float] = None, softcap: float = 0.0,
                            window: int = 0, causal: bool = True, return_lse: bool = False,
                            out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, sinks: int = 0,
                            k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
    """Attention of the new tokens' queries q [T, Hq, D] over their sequences' paged caches
    [pages, page_size, Hkv, D] (bf16 or fp16, D 64, 128 or 256, Hq a multiple of Hkv); returns o
    [T, Hq, D], or (o, lse [T, Hq] fp32) with ``return_lse``.

    Sequence b's new tokens (rows ``cu_seqlens[b] ..``) are the last of those it holds, already
    appended.  A row sees the tokens up to its own (``causal``) and, with ``window``, only the
    last ``window`` of them; ``softcap`` bounds the scores by ``softcap * tanh(x / softcap)`` (0: no
    bound); ``scale`` defaults to 1/sqrt(D) (None or 0).  Neither may be negative.  ``out`` must not share memory with q.

    ``sinks`` first tokens of a sequence stay visible beside a window (without one all are).  Caches of 8
    bits (``torch.float8_e4m3fn``) come with the ``k_scale`` and ``v_scale`` that ``kv_append_paged`` wrote; the
    result is that of a cache of their values (in fp16 those over 65,504 are infinite)."""
    return _attention("prefill", q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size,
                      last_page_len, scale, softcap, window, causal, return_lse, out, workspace, sinks, k_scale, v_scale)


def attention_decode_paged(q, k_cache, v_cache, page_indices, page_indptr, page_size: int, last_page_len,
                           scale: Optional[float] = None, softcap: float = 0.0, window: int = 0,
                           return_lse: bool = False, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, sinks: int = 0,
                           k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
    """``attention_prefill_paged`` for one token per sequence: q [B, Hq, D], row b at the last
    position of sequence b (a sequence without a page gives zeros and an lse of -inf).  ``out`` may
    be q."""
    return _attention("decode", q, None, k_cache, v_cache, page_indices, page_indptr, page_size,
                      last_page_len, scale, softcap, window, True, return_lse, out, workspace, sinks, k_scale, v_scale)
