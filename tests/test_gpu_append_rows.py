"""The append takes no more rows than the call gives it: sequences whose end lies past them (a batch cut short) have
their rows up to there written, in 16 bits and in 8, and the rows that follow in memory are not read."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import quantised

pytestmark = pytest.mark.gpu
DEV, BF, E4M3 = "cuda", torch.bfloat16, torch.float8_e4m3fn
MOST = 1.875 * 2.0 ** 127


def lib():
    import paged_recurrent_state_amd as m
    return m


@pytest.mark.parametrize("rows", [1, 2, 17, 39, 61])
@pytest.mark.parametrize("sizes", [[70], [3, 70, 5], [20, 0, 41, 9], [1] * 80, [2] * 40])
def test_a_batch_cut_short(rows, sizes):
    m, H, D, page = lib(), 2, 64, 32
    past = [(7 * i) % 40 for i in range(len(sizes))]
    c = au.batch([a + b for a, b in zip(sizes, past)], page, H, D, BF, 5, DEV)
    cu = [0] + np.cumsum(sizes).tolist()
    x = au.queries(cu[-1], 2 * H + 3, D, BF, 6, DEV)
    x[rows:] *= 1000.0  # (rows that the call does not have: they would raise every scale)
    k, v, q = x[:rows, :H], x[:rows, H:2 * H], x[:rows, 2 * H:]
    rest = {n: c[n] for n in ("page_indices", "page_indptr", "page_size", "last_page_len")}
    tab = m.rope_table(128, 32, device=DEV)
    tab[:, :16], tab[:, 16:] = 1.0, 0.0  # (keys and queries as they are)
    for coded in (False, True):
        kv = {n: (torch.randn(c[n].shape, device=DEV) * 100).to(E4M3 if coded else BF) for n in ("k_cache", "v_cache")}
        sc = {n: torch.full((kv["k_cache"].shape[0], 2, H), 0.5, device=DEV) for n in ("k_scale", "v_scale")} if coded else {}
        codes = {n: (y.view(torch.uint8).cpu().view(E4M3).double() if coded else y.cpu().double()).numpy().copy() for n, y in kv.items()}
        scales = {n: y.cpu().double().numpy().copy() for n, y in sc.items()}
        got_q = m.kv_append_paged(k, v, au.i32(cu, DEV), **kv, **rest, **sc, table=tab, q=q)
        torch.cuda.synchronize()
        assert torch.equal(got_q, q.contiguous())
        # the rows there are, at the places they have in the whole sequences
        new = [max(0, min(rows, cu[b + 1]) - cu[b]) for b in range(len(sizes))]
        lens = [past[b] + new[b] for b in range(len(sizes))]
        ids, ptr = rest["page_indices"].tolist(), rest["page_indptr"].tolist()
        for name, y in (("k", k), ("v", v)):
            want = codes[name + "_cache"]
            if coded:
                quantised.append(want, scales[name + "_scale"], au.f64(y), new, lens, ids, ptr, page, 16, MOST)
                assert np.array_equal(sc[name + "_scale"].cpu().double().numpy(), scales[name + "_scale"])
                got = kv[name + "_cache"].view(torch.uint8).cpu().view(E4M3).double().numpy()
            else:
                for b in range(len(sizes)):
                    for i in range(new[b]):
                        p = past[b] + i
                        want[ids[ptr[b] + p // page], p % page] = au.f64(y[cu[b] + i])
                got = kv[name + "_cache"].cpu().double().numpy()
            assert np.array_equal(got, want, equal_nan=True)
