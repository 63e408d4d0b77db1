"""Inputs and error bounds shared by the tests of the attention layers."""

from __future__ import annotations

import numpy as np
import torch

from oracle import attention as oatt

NAN = float("nan")
# Largest relative error of one rounding to nearest: half the spacing above a power of two, which
# is 2^-7, 2^-10 and 2^-23 of it (8, 11 and 24 significant bits).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least step


def batch(lens, page_size, heads, dim, dtype, seed, device="cpu", heads_first=False, spare=2, gain=1.0):
    """Page table and caches of sequences of ``lens`` tokens (0: a sequence without a page); every
    slot that no sequence holds is NaN.  Page ids are a seeded permutation."""
    gen = torch.Generator().manual_seed(seed)
    pages = [-(-n // page_size) for n in lens]
    total = sum(pages) + spare
    ids = torch.randperm(total, generator=gen).to(torch.int32)[:sum(pages)]
    ptr = [0]
    for n in pages:
        ptr.append(ptr[-1] + n)
    lpl = [n - (k - 1) * page_size if k else 0 for n, k in zip(lens, pages)]
    kv = torch.full((2, total, page_size, heads, dim), NAN, dtype=dtype)
    for b in range(len(lens)):
        for j, (p, i) in enumerate(oatt.slots(ids.tolist(), ptr, lpl, page_size, b)):
            kv[:, p, i] = (torch.randn(2, heads, dim, generator=gen) * gain).to(dtype)
    if heads_first:
        kv = kv.transpose(2, 3).contiguous().transpose(2, 3)
    i32 = dict(dtype=torch.int32, device=device)
    kv = kv.to(device)
    return dict(k_cache=kv[0], v_cache=kv[1], page_indices=ids.to(device),
                page_indptr=torch.tensor(ptr, **i32), page_size=page_size,
                last_page_len=torch.tensor(lpl, **i32))


def queries(T, heads, dim, dtype, seed, device="cpu", gain=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, heads, dim, generator=gen) * gain).to(dtype).to(device)


def i32(x, device="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def f64(x):
    return x.detach().float().cpu().double().numpy()


def attention_bounds(ref, dim, dtype, softcap=0.0):
    """Largest error of o and lse that the arithmetic allows, value by value.

    A score is a sum of D exact products in fp32: off by at most D 2^-24 sum |q_d k_d| (times
    the scale), and its scaling, the tanh and the exponential's argument round to 2^-22 of the
    largest score or cap.  A weight e^{x - m} is off by that much relatively (twice: the quotient's
    numerator and denominator), the exponential by 2^-22, its rounding to the element type by
    UNIT; the sums over the keys round to 2^-20 at the lengths tested.  o then rounds once."""
    o, lse, mag, spread, reach = ref
    u = UNIT[dtype]
    score = dim * 2.0 ** -24 * spread + 2.0 ** -21 * (1.0 + reach + softcap)
    eo = mag * (u + 2 * score[..., None] + 2.0 ** -19) * (1 + u) + u * np.abs(o) + TINY[dtype]
    return eo, score + 2.0 ** -20


def check_attention(got_o, got_lse, ref, dim, dtype, softcap=0.0, what=""):
    eo, el = attention_bounds(ref, dim, dtype, softcap)
    o, lse = ref[0], ref[1]
    x = f64(got_o)
    assert np.isfinite(x).all(), f"{what}: non-finite output"
    worst = float((np.abs(x - o) / eo).max()) if x.size else 0.0
    assert worst <= 1.0, f"{what}: output error {worst:.2f} times its bound"
    if got_lse is not None:
        y = f64(got_lse)
        none = np.isneginf(lse)
        assert (np.isneginf(y) == none).all(), f"{what}: lse of rows that see nothing"
        d = np.abs(y[~none] - lse[~none]) / el[~none]
        assert not d.size or d.max() <= 1.0, f"{what}: lse error {d.max():.2f} times its bound"
    return worst


def rotation_bounds(x, dtype, rot, tab):
    """|error| of a rotated value: two products and a sum in fp32 of an exact input and a table
    value (2^-22 of |a c| + |b s| <= the pair's norm times the table's magnitude), rounded once."""
    mag = float(np.sqrt((np.asarray(tab, dtype=np.float64) ** 2).max() * 2)) if tab.size else 1.0
    top = np.abs(x).max(axis=-1, keepdims=True) * 2 * max(mag, 1.0)
    return top * (2.0 ** -22), UNIT[dtype]
