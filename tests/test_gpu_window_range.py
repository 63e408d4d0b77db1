"""Windows past 32 bits leave nothing out, and negative ones of any size are refused."""

import pytest
import torch

import attention_util as au

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def calls(coded):
    import paged_recurrent_state_amd as m
    c = au.batch([300, 41], 16, 2, 64, BF, 0, DEV)
    if coded:
        sc = torch.ones(c["k_cache"].shape[0], 1, 2, device=DEV)
        c = {**c, "k_scale": sc, "v_scale": sc.clone(), **{n: c[n].to(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")}}
    q, cu = au.queries(50, 4, 64, BF, 1, DEV), au.i32([0, 30, 50], DEV)
    return (lambda **kw: m.attention_prefill_paged(q, cu, **c, return_lse=True, **kw),
            lambda **kw: m.attention_decode_paged(q[:2], **c, return_lse=True, **kw))


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("sinks", [0, 4])
def test_windows(coded, sinks):
    import paged_recurrent_state_amd as m
    for call in calls(coded):
        want = call()
        for window in (1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 33) - 7, 1 << 64):
            assert all(torch.equal(a, b) for a, b in zip(call(window=window, sinks=sinks), want)), window
        for window in (-1, -(1 << 31), -(1 << 32) + 5, -(1 << 32), -(1 << 70)):
            with pytest.raises(m.GDNError, match="window"):
                call(window=window, sinks=sinks)
