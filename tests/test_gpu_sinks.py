"""First tokens that stay visible beside a window, over 16-bit caches, against the fp64
oracle: their number against the window, the history and the pages, chunks and
decoded tokens, shares that end among them, layouts, values that are not finite."""

import numpy as np
import pytest
import torch

import attention_util as au
from test_gpu_attention import case, check_prefill, lib, oracle_of, run_prefill

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def check_decode(lens, page, H, G, D, dtype, seed, **kw):
    q, _, c = case([1 if n else 0 for n in lens], [max(0, n - 1) for n in lens], page, H, G, D, dtype, seed)
    q = au.queries(len(lens), H * G, D, dtype, seed + 1, DEV)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True, **kw)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c, **kw), D, dtype, kw.get("softcap", 0.0))


@pytest.mark.parametrize("window", [1, 3, 32, 64, 65, 300])
@pytest.mark.parametrize("sinks", [1, 4, 31, 32, 33, 64, 100, 1000])
def test_windows(window, sinks):
    check_prefill([70, 1, 0, 200], [500, 130, 64, 0], 16, 2, 2, 128, BF, 10, window=window, sinks=sinks)
    check_decode([570, 131, 0, 64, 1, 33, 2], 16, 2, 2, 128, BF, 11, window=window, sinks=sinks)


@pytest.mark.parametrize("D,dtype", [(64, HF), (64, BF), (128, HF), (256, BF), (256, HF)])
@pytest.mark.parametrize("page", [1, 5, 48, 100, 896])
def test_heads_types_and_pages(D, dtype, page):
    check_prefill([130, 40], [600, 5], page, 2, 3, D, dtype, 20, window=90, sinks=7)
    check_decode([730, 45, 91, 97, 98], page, 2, 3, D, dtype, 21, window=90, sinks=7)


@pytest.mark.parametrize("cap", [20.0, 100.0])
def test_caps_and_layout(cap):
    for D, dtype in ((64, HF), (128, BF), (256, BF)):
        check_prefill([130], [300], 16, 2, 2, D, dtype, 30, heads_first=True, gain=3.0, window=50, sinks=70, softcap=cap)
        check_decode([430, 20], 16, 2, 2, D, dtype, 31, window=50, sinks=70, softcap=cap)


def test_every_distance_between_sinks_and_window():
    """Tiles of both, one, or neither, and rows whose window begins inside them."""
    for past in range(0, 140, 9):
        check_prefill([66], [past], 16, 1, 1, 64, BF, 40 + past, window=33, sinks=20)
        check_decode([past + 1, past + 30, past + 66], 16, 1, 1, 64, BF, 41 + past, window=33, sinks=20)


def test_not_causal():
    check_prefill([100], [150], 16, 2, 1, 128, BF, 50, window=40, sinks=5, causal=False)


def test_without_a_window_or_sinks_nothing_changes():
    q, cu, c = case([60, 3], [200, 10], 16, 2, 2, 128, BF, 60)
    a = run_prefill(q, cu, c)
    b = run_prefill(q, cu, c, sinks=9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = run_prefill(q, cu, c, window=50)
    b = run_prefill(q, cu, c, window=50, sinks=0)
    assert torch.equal(a[0], b[0])
    # sinks and window that leave nothing out
    a = run_prefill(q, cu, c)
    b = run_prefill(q, cu, c, window=100, sinks=200)
    au.check_attention(b[0], b[1], oracle_of(q, cu, c), 128, BF)
    assert au.f64(a[0] - b[0]).max() < 0.02


def test_long_batches():
    """Shares that start or end among the first tokens' tiles, joined from parts; runs of a few tiles each."""
    new, past = [300, 1, 40, 513], [3000, 5000, 0, 900]
    for D, dtype in ((64, HF), (128, BF), (256, BF)):
        check_prefill(new, past, 48, 2, 4, D, dtype, 70, window=700, sinks=130)
    check_decode([(i * 331) % 5000 for i in range(60)], 48, 2, 4, 128, BF, 71, window=700, sinks=130)
    check_decode([9000], 16, 1, 2, 128, BF, 72, window=4000, sinks=2000)


def test_more_queries_than_tiles_listed_by_a_workgroup():
    """Over 256 tiles of rows: the plan is a kernel of its own."""
    check_prefill([1] * 300 + [2] * 40, [(i * 7) % 300 for i in range(340)], 16, 1, 2, 64, BF, 75, window=20, sinks=3)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_infinities_among_the_sinks(D, dtype):
    """An infinite value at a first token reaches every row, one in the gap those that see it."""
    new, past, window, sinks = [90], [400], 64, 5
    q, cu, c = case(new, past, 16, 1, 2, D, dtype, 80)
    first, gap = int(c["page_indices"][0]), int(c["page_indices"][25])  # tokens 0 .., 400 ..
    c["v_cache"][first, 2, 0, 7] = float("inf")
    c["v_cache"][gap, 3, 0, 9] = -float("inf")  # token 403: rows 403 .. 466
    o, lse = run_prefill(q, cu, c, window=window, sinks=sinks)
    assert torch.isposinf(o[:, :, 7]).all() and torch.isfinite(lse).all()
    sees = torch.zeros(90, dtype=torch.bool, device=DEV)
    sees[3:3 + window] = True
    assert torch.isneginf(o[sees][:, :, 9]).all() and torch.isfinite(o[~sees][:, :, 9]).all()
    rest = [d for d in range(D) if d not in (7, 9)]
    assert torch.isfinite(o[:, :, rest]).all()
    o = lib().attention_decode_paged(q[-1:].contiguous(), **c, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert torch.isposinf(o[:, :, 7]).all() and torch.isfinite(o[:, :, rest + [9]]).all()


def test_nan_between_sinks_and_window_is_not_read_into_any_row():
    q, cu, c = case([64], [600], 16, 2, 1, 128, BF, 90)
    ref, want = run_prefill(q, cu, c, window=100, sinks=10), oracle_of(q, cu, c, window=100, sinks=10)
    for i in range(1, 25):  # tokens 16 .. 399
        c["k_cache"][int(c["page_indices"][i])] = float("nan")
        c["v_cache"][int(c["page_indices"][i])] = float("nan")
    got = run_prefill(q, cu, c, window=100, sinks=10)
    # (NaN beside the sinks in their tile: the share is computed again, with other references and roundings)
    au.check_attention(*ref, want, 128, BF)
    au.check_attention(*got, want, 128, BF)
    a = lib().attention_decode_paged(q[-1:].contiguous(), **c, window=100, sinks=10)
    torch.cuda.synchronize()
    assert torch.isfinite(a).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(100 + seed)
    D, dtype = int(r.choice([64, 128, 256])), [BF, HF][int(r.integers(2))]
    page, B = int(r.choice([1, 5, 16, 64, 100])), int(r.integers(1, 5))
    new, past = [int(x) for x in r.integers(0, 150, B)], [int(x) for x in r.integers(0, 700, B)]
    kw = dict(window=int(r.integers(1, 300)), sinks=int(r.choice([1, 4, 20, 64, 65, 200])), softcap=float(r.choice([0.0, 20.0])))
    H, G = int(r.integers(1, 4)), int(r.integers(1, 6))
    check_prefill(new, past, page, H, G, D, dtype, 200 + seed, bool(r.integers(2)), **kw)
    check_decode([p + 1 for p in past], page, H, G, D, dtype, 300 + seed, **kw)


@pytest.mark.parametrize("sinks", [-1, (1 << 30) + 1, 1 << 32, (1 << 32) + 4])
def test_numbers_of_sinks_past_the_calls_range_are_refused(sinks):
    q, cu, c = case([5], [20], 16, 1, 1, 64, BF, 95)
    with pytest.raises(lib().GDNError, match="sinks"):
        lib().attention_prefill_paged(q, au.i32(cu, DEV), **c, window=4, sinks=sinks)
    with pytest.raises(lib().GDNError, match="sinks"):
        lib().attention_decode_paged(q[:1], **c, window=4, sinks=sinks)
