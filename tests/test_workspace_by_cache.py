"""What an attention call needs of a workspace goes by the type of its cache: 16-bit calls no more than
they would without the 8-bit ones, in the library and in the binding."""

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn
from paged_recurrent_state_amd import _attention, _lib
from paged_recurrent_state_amd._lib import _AttentionC

BF, HF, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
HEADS = [(1, 1), (8, 2), (32, 8), (7, 1), (8, 1), (24, 2), (16, 1), (64, 2)]


def parts(waves, rows, dim):
    """Bytes of two parts a wave, each with `rows` outputs and two sums a row, and 16 bytes of what they belong to."""
    return waves * (2 * rows * (dim + 2) * 4 + 16)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_needs(heads, dim):
    Hq, Hk = heads
    for T, B in ((0, 0), (1, 1), (7, 2), (512, 512), (3000, 5)):
        any_, codes = (gdn.attention_workspace_size(T, B, Hq, Hk, dim, *x) for x in ((), (E4M3,)))
        plain = gdn.attention_workspace_size(T, B, Hq, Hk, dim, BF)
        assert plain == gdn.attention_workspace_size(T, B, Hq, Hk, dim, HF) and any_ == max(plain, codes)
        if Hq // Hk <= 7:
            assert codes <= plain
    # one token: the waves' parts, and nothing else, with the compute units of the first line
    cus = gdn.attention_workspace_size(1, 1, Hq, Hk, 64, BF) // parts(8, 16, 64)
    per_cu = {64: (2, 3), 128: (2, 3), 256: (1, 2)}[dim]
    assert gdn.attention_workspace_size(1, 1, Hq, Hk, dim, BF) == parts(4 * cus * per_cu[0], 16, dim)
    assert gdn.attention_workspace_size(1, 1, Hq, Hk, dim, E4M3) >= parts(4 * cus * per_cu[1], min(16, Hq // Hk), dim)


def test_the_binding_asks_by_the_cache():
    for Hq, Hk in HEADS:
        for dim in (64, 128, 256):
            for coded, dtype in ((False, BF), (True, E4M3)):
                assert _attention._workspace_size(5, 2, Hq, Hk, dim, 0, coded) == gdn.attention_workspace_size(5, 2, Hq, Hk, dim, dtype)


def test_bad_arguments():
    for bad in (torch.float32, torch.uint8, torch.float8_e5m2, "bf16"):
        with pytest.raises(TypeError):
            gdn.attention_workspace_size(1, 1, 8, 2, 64, bad)
    assert _lib.load().gdn_attention_workspace_size_ext(_AttentionC(8, 3, 64, 0, 0.0, 0.0, 0, 1), 1, 5, 2) == 0
    assert gdn.attention_workspace_size(-1, 1, 8, 2, 64, E4M3) == 0


def codes_of(c):
    """The batch's cache as codes under scales of one (NaN where no sequence holds a token)."""
    sc = torch.ones(c["k_cache"].shape[0], 1, c["k_cache"].shape[2], device="cuda")
    kv = {n: c[n].to(E4M3) for n in ("k_cache", "v_cache")}
    return {**c, **kv, "k_scale": sc, "v_scale": sc.clone()}


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 2), (11, 1), (12, 1), (16, 1), (40, 2)])
def test_calls_take_what_their_cache_needs(dim, heads):
    """A buffer of exactly that size, with what lies behind it left as it was; groups of one to three blocks of rows, and
    runs long enough to be joined from many waves' parts."""
    dev, (Hq, Hk) = "cuda", heads
    c = au.batch([50, 9000, 700], 16, Hk, dim, BF, 0, dev)
    q, cu = au.queries(3, Hq, dim, BF, 1, dev), au.i32([0, 1, 2, 3], dev)
    sixteen = {n: codes_of(c)[n].to(BF) for n in ("k_cache", "v_cache")}
    for coded, args in ((False, {**c, **sixteen}), (True, codes_of(c))):
        n = gdn.attention_workspace_size(3, 3, Hq, Hk, dim, E4M3 if coded else BF)
        ws = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device=dev)
        for call in (lambda w: gdn.attention_decode_paged(q, **args, workspace=w, return_lse=True),
                     lambda w: gdn.attention_prefill_paged(q, cu, **args, workspace=w, return_lse=True)):
            ref, got = call(None), call(ws[:n])
            assert all(torch.equal(a, b) for a, b in zip(ref, got)) and (ws[n:] == 0x5a).all()
            with pytest.raises(ValueError, match="workspace"):
                call(ws[:n - 1])
        if not coded:
            plain = gdn.attention_decode_paged(q, **args)
    # the same values in 8 bits: the runs' ends differ, the rounding of the output is the same
    got = gdn.attention_decode_paged(q, **codes_of(c))
    o, lse, *rest = au.oatt.attention_paged(au.f64(q), cu.tolist(), au.f64(sixteen["k_cache"]), au.f64(sixteen["v_cache"]),
                                            c["page_indices"].tolist(), c["page_indptr"].tolist(), 16, c["last_page_len"].tolist())
    for x in (plain, got):
        au.check_attention(x, None, (o, lse, *rest), dim, BF)
