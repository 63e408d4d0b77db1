"""ctypes binding of the attention layers' entry points (include/gdn_attention.h):
rotary positions, the append to a paged key/value cache, and attention over it.

Argument marshalling only, as in ``_lib``: every step runs in the HIP library on
the tensors' device, on torch's current stream, and there is no fallback.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple

import torch

from ._lib import (GDN_INDEX_INT32, GDN_INDEX_INT64, _AttentionC, _CacheC, _check, _need, _RopeC, _RowsC,
                   _ScalingC, _workspace, load)
from ._lib import _stream as _stream_of_device

# element types (GDN_TYPE_*)
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


def _stream(dev: torch.device):
    """torch's current stream on ``dev``: its handle alone, since at small sizes a
    ``torch.cuda.Stream`` object would cost as much as the kernel."""
    if dev.type != "cuda" or dev.index is None:
        return _stream_of_device(dev)
    return torch._C._cuda_getCurrentRawStream(dev.index)


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
    _check(lib.gdn_rope_table(sc, table.data_ptr(), int(positions), int(rot_dim), stream))
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
    ``q_out`` or ``k_out`` exclude each other, and the table has no gradient."""
    # (asked first and without a call: at one token the host's time is all there is)
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


def _rope_rows(q, k, table, positions, interleaved, transposed, q_out, k_out):
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
    _check(lib.gdn_rope(rp, code, D, Hq, Hk, T, positions.data_ptr(),
                        GDN_INDEX_INT64 if positions.dtype == torch.int64 else GDN_INDEX_INT32,
                        qr, kr, qo, ko, stream))
    return q_out, k_out


def rope_backward(dq, dk, table, positions, interleaved: bool = False,
                  q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of ``rope``'s inputs from those of its outputs (the transposed map)."""
    return rope(dq, dk, table, positions, interleaved, True, q_out, k_out)


def kv_append_paged(k, v, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size: int,
                    last_page_len, table: Optional[torch.Tensor] = None, interleaved: bool = False,
                    q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    ) -> Optional[torch.Tensor]:
    """Write the new tokens' k and v [T, Hkv, D] to the paged caches [pages, page_size, Hkv, D]
    (any strides, the last dimension dense), in one launch (no gradient: a serving call, as the
    attention calls on these caches).

    ``table`` (``rope_table``) rotates the keys on the way, and ``q`` [T, Hq, D], when given, into
    ``q_out`` (returned; a new tensor unless given).  The page table is the one after the
    append; ``cu_seqlens`` [B + 1] gives each sequence's new tokens, None one token each."""
    lib = load()
    code, dev = _dtype(k, "k"), k.device
    stream = _stream(dev)
    kr = _rows(k, "k", k.dtype, dev)
    T, Hk, D = k.shape
    vr = _rows(v, "v", k.dtype, dev, Hk, T, D)
    cache = _cache(k_cache, v_cache, page_indices, page_indptr, int(page_size), last_page_len, k.dtype, dev, D)
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
    _check(lib.gdn_kv_append_paged(rp, code, D, Hq, Hk, cu, T, kr, vr, cache, qr, qo, stream))
    return q_out


@lru_cache(maxsize=256)
def _workspace_size(total_tokens: int, num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                    device: int) -> int:
    d = _AttentionC(num_q_heads, num_kv_heads, head_dim, 0, 0.0, 0.0, 0, 1)
    return int(load().gdn_attention_workspace_size(d, total_tokens, num_seqs))


def attention_workspace_size(total_tokens: int, num_seqs: int, num_q_heads: int, num_kv_heads: int,
                             head_dim: int) -> int:
    """Bytes either attention call needs for at most that many query rows and sequences."""
    d = _AttentionC(num_q_heads, num_kv_heads, head_dim, 0, 0.0, 0.0, 0, 1)
    return int(load().gdn_attention_workspace_size(d, int(total_tokens), int(num_seqs)))


def _attention(fn, q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size, last_page_len,
               scale, softcap, window, causal, return_lse, out, workspace):
    lib = load()
    code, dev = _dtype(q, "q"), q.device
    stream = _stream(dev)
    qr = _rows(q, "q", q.dtype, dev)
    T, Hq, D = q.shape
    cache = _cache(k_cache, v_cache, page_indices, page_indptr, int(page_size), last_page_len, q.dtype, dev, D)
    # (the library takes what is not positive for its defaults)
    scale, softcap = 0.0 if scale is None else float(scale), 0.0 if softcap is None else float(softcap)
    if scale < 0.0 or softcap < 0.0:
        raise ValueError(f"scale and softcap must not be negative, got {scale} and {softcap}")
    d = _AttentionC(Hq, k_cache.shape[2], D, code, scale, softcap, int(window), bool(causal))
    if out is None:
        out, o = _dense((T, Hq, D), q.dtype, dev)
    else:
        o = _rows(out, "out", q.dtype, dev, Hq, T, D)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if return_lse else None
    ws = _workspace(workspace, _workspace_size(T, cache.num_seqs, Hq, k_cache.shape[2], D, dev.index), dev)
    tail = (cache, o, lse.data_ptr() if return_lse else None, ws.data_ptr(), ws.numel() * ws.element_size(),
            stream)
    if fn == "prefill":
        rc = lib.gdn_attention_prefill_paged(d, qr, _cu(cu_seqlens, cache.num_seqs, dev), T, *tail)
    else:
        if T != cache.num_seqs:
            raise ValueError(f"q must have one row per sequence ({cache.num_seqs}), got {T}")
        rc = lib.gdn_attention_decode_paged(d, qr, *tail)
    _check(rc)
    return (out, lse) if return_lse else out


def attention_prefill_paged(q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size: int,
                            last_page_len, scale: Optional[float] = None, softcap: float = 0.0,
                            window: int = 0, causal: bool = True, return_lse: bool = False,
                            out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Attention of the new tokens' queries q [T, Hq, D] over their sequences' paged caches
    [pages, page_size, Hkv, D] (bf16 or fp16, D 64, 128 or 256, Hq a multiple of Hkv); returns o
    [T, Hq, D], or (o, lse [T, Hq] fp32) with ``return_lse``.

    Sequence b's new tokens (rows ``cu_seqlens[b] ..``) are the last of those it holds, already
    appended.  A row sees the tokens up to its own (``causal``) and, with ``window``, only the
    last ``window`` of them; ``softcap`` bounds the scores by ``softcap * tanh(x / softcap)`` (0: no
    bound); ``scale`` defaults to 1/sqrt(D) (None or 0).  Neither may be negative.  ``out`` must not share memory with q."""
    return _attention("prefill", q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size,
                      last_page_len, scale, softcap, window, causal, return_lse, out, workspace)


def attention_decode_paged(q, k_cache, v_cache, page_indices, page_indptr, page_size: int, last_page_len,
                           scale: Optional[float] = None, softcap: float = 0.0, window: int = 0,
                           return_lse: bool = False, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """``attention_prefill_paged`` for one token per sequence: q [B, Hq, D], row b at the last
    position of sequence b (a sequence without a page gives zeros and an lse of -inf).  ``out`` may
    be q."""
    return _attention("decode", q, None, k_cache, v_cache, page_indices, page_indptr, page_size,
                      last_page_len, scale, softcap, window, True, return_lse, out, workspace)
