"""Values that cannot be stored as they are (NaN, infinities, magnitudes next to the type's largest) on every way
through the quantising append: blocks of up to four new tokens, which a row's lanes take (decoded ones among them),
of one, two and all waves, and of rows that are read twice; pieces of 16 and of 4 bytes; blocks opened and joined.
Odd values lie in some heads only, so that waves that wait together disagree.  Codes and scales bit for bit."""

import numpy as np
import pytest
import torch

import attention_util as au
from test_gpu_quantised import BF, DEV, HF, MOST, Cache, codes_of, half_step
from oracle import attention as oatt
from oracle import norms

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def odd_rows(T, H, D, dtype, seed, starts, narrow):
    """[T, H, D] rows: in the tokens from each start on, every third head has NaN, infinities or the type's largest
    values, in another order for each start, and the heads between them none.  narrow: rows at multiples of 4 bytes."""
    x = au.queries(T, H, D, dtype, seed, DEV)
    most = torch.finfo(dtype).max
    for j, t in enumerate(starts):
        for h in range(j % 3, H, 3):
            kind = (j + h) % 5
            if kind == 0:
                x[t, h, j % D] = NAN
            elif kind == 1:
                x[t, h, (3 * j) % D], x[t, h, D - 1] = INF, -INF
            elif kind == 2:
                x[t, h, (5 * j) % D] = most
            elif kind == 3:
                x[t, h] = NAN  # the whole row
            else:
                x[t, h, 0], x[t, h, D // 2], x[t, h, D - 1] = -most, NAN, INF
    if narrow:
        flat = torch.empty(T * H * D + 2, dtype=dtype, device=DEV)
        flat[2:].view(T, H, D).copy_(x)
        x = flat[2:].view(T, H, D)
    return x


def check(new, past, page, block, H, D, dtype, seed, starts, narrow=False, decode=False):
    lens = [a + b for a, b in zip(new, past)]
    a = Cache(lens, page, block, H, D, seed)
    T, cu = sum(new), [0] + np.cumsum(new).tolist()
    k, v = (odd_rows(T, H, D, dtype, seed + i, starts[i:], narrow) for i in (0, 1))
    a.append(k, v, None if decode else au.i32(cu, DEV))
    torch.cuda.synchronize()
    for n, x in (("k", k), ("v", v)):
        a.expect(n, au.f64(x), new, lens, MOST[dtype])
        a.check(n)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("narrow", [False, True])
def test_decoded_tokens(dtype, D, narrow):
    """One token each, opening a block or joining one, whose scale grows (to the largest there is) or stays."""
    past = [0, 1, 15, 16, 31, 40, 47, 48] * 3
    check([1] * 24, past, 48, 16, 4, D, dtype, 10 + D, list(range(0, 24, 2)), narrow, decode=True)
    check([1] * 24, past, 48, 48, 4, D, dtype, 11 + D, list(range(24)), narrow)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("narrow", [False, True])
def test_few_tokens(dtype, D, narrow):
    new = [2, 3, 4, 4, 1, 0, 4, 2, 3, 4]
    check(new, [0, 14, 13, 30, 47, 5, 44, 7, 16, 63], 64, 16, 5, D, dtype, 20 + D, list(range(0, 27, 2)), narrow)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("rows", [5, 12, 40, 70, 100, 140, 300, 700])
def test_blocks_of_every_length(rows, D, dtype, narrow):
    """A lane keeps four rows: a wave 256 (heads of 64, pieces of 16 bytes) down to 4 (of 256, pieces of 4 bytes)."""
    starts = [0, rows - 1, rows // 2, rows, rows + rows // 3]
    check([rows, rows], [0, 190], 896, 896, 5, D, dtype, 30 + rows + D, starts, narrow)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_of_all_lengths_together(D):
    new = [3, 1, 300, 20, 2, 0, 130, 70, 17, 1100, 5, 40, 9, 33, 257, 64, 128, 16, 1, 1]
    T = sum(new)
    check(new, [(i * 37) % 120 for i in range(len(new))], 896, 896, 6, D, BF, 40 + D, list(range(0, T, 23)))
    check(new, [(i * 37) % 120 for i in range(len(new))], 896, 64, 6, D, HF, 41 + D, list(range(0, T, 7)))


def test_normed_and_turned_rows_with_odd_values():
    """A row with one of them is NaN as a whole after the norm, and counts for no scale."""
    import paged_recurrent_state_amd as m
    D, H, dtype = 128, 3, BF
    tab = m.rope_table(2000, 64, device=DEV)
    w = torch.rand(D, device=DEV) + 0.5
    for new in ([1, 1, 1], [3, 2, 4], [40, 100, 300]):
        past = [5, 17, 60]
        lens = [a + b for a, b in zip(new, past)]
        T, pos = sum(new), [p + i for n, p in zip(new, past) for i in range(n)]
        a = Cache(lens, 896, 448, H, D, 50)
        x = au.queries(T, 2 * H, D, dtype, 51, DEV)
        x[0, 0, 3], x[T // 2, 1, 5], x[T - 1, 2] = NAN, INF, NAN
        k, v = x[:, :H], x[:, H:]
        a.append(k, v, au.i32([0] + np.cumsum(new).tolist(), DEV), table=tab, k_norm=w)
        torch.cuda.synchronize()
        with np.errstate(invalid="ignore"):
            y = norms.norm_rope(au.f64(k), au.f64(w), au.f64(tab), pos, 1e-6)
        a.expect("k", y, new, lens, MOST[dtype])
        a.expect("v", au.f64(v), new, lens, MOST[dtype])
        a.check("v")
        assert np.array_equal(a.s["k_scale"].cpu().double().numpy(), a.scales["k"])
        got = codes_of(a.c["k_cache"])
        assert np.array_equal(np.isnan(got), np.isnan(a.codes["k"]))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("D,rot,normed", [(128, 128, False), (64, 32, True), (256, 64, True)])
def test_computed_keys_are_rounded_once(dtype, near, D, rot, normed):
    """Code times scale is within half a step of the value in 64 bits, where the step is that of the value, and the
    value in 32 bits is off by 2^-19 of twice its row's largest (as the append's queries)."""
    import paged_recurrent_state_amd as m
    new, past, H, page, block = [30, 1, 0, 5, 300], [3, 40, 2, 0, 64], 3, 64, 32
    lens = [a + b for a, b in zip(new, past)]
    a = Cache(lens, page, block, H, D, 60)
    T, pos = sum(new), [p + i for n, p in zip(new, past) for i in range(n)]
    kv = au.queries(T, 2 * H, D, dtype, 61, DEV)
    k, v = kv[:, :H], kv[:, H:]
    w = torch.rand(D, device=DEV) + 0.5
    tab = m.rope_table(400, rot, device=DEV)
    a.append(k, v, au.i32([0] + np.cumsum(new).tolist(), DEV), table=tab, interleaved=near,
             **(dict(k_norm=w, eps=1e-5, norm_offset=0.25) if normed else {}))
    torch.cuda.synchronize()
    want = (norms.norm_rope(au.f64(k), au.f64(w), au.f64(tab), pos, 1e-5, 0.25, near) if normed
            else oatt.rotate(au.f64(k), au.f64(tab), pos, near))
    codes, scale = codes_of(a.c["k_cache"]), a.s["k_scale"].cpu().double().numpy()
    ids, ptr, t = a.where["page_indices"].tolist(), a.where["page_indptr"].tolist(), 0
    for b, n in enumerate(new):
        for i in range(past[b], lens[b]):
            p, off = ids[ptr[b] + i // page], i % page
            s = scale[p, off // block][:, None]
            err = np.abs(want[t]).max(axis=-1, keepdims=True) * 2 * 2.0 ** -19
            # (the step of the value in 32 bits, which may lie in the next binade up)
            step = half_step((np.abs(want[t]) + err) / s) * s
            assert (np.abs(codes[p, off] * s - want[t]) <= step + err).all(), (b, i)
            t += 1
