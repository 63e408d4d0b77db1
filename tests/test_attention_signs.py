"""Scales and caps of the attention calls: none may be negative, 0 and None are the defaults."""

import math

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_signs():
    c = au.batch([5, 90], 16, 2, 64, BF, 0, DEV)
    q, cu = au.queries(2, 4, 64, BF, 1, DEV), au.i32([0, 1, 2], DEV)
    for call in (lambda **kw: gdn.attention_decode_paged(q, **c, return_lse=True, **kw),
                 lambda **kw: gdn.attention_prefill_paged(q, cu, **c, return_lse=True, **kw)):
        for kw in (dict(scale=-0.125), dict(softcap=-30.0), dict(scale=-1, softcap=5.0), dict(scale=-math.inf)):
            with pytest.raises(ValueError, match="negative"):
                call(**kw)
        for kw in (dict(scale=math.nan), dict(softcap=math.nan), dict(scale=math.inf), dict(softcap=math.inf)):
            with pytest.raises(gdn.GDNError):
                call(**kw)
        want = call()
        for kw in (dict(scale=None), dict(scale=0), dict(scale=1 / 8), dict(softcap=0), dict(softcap=None), dict(scale=-0.0)):
            assert all(torch.equal(a, b) for a, b in zip(call(**kw), want)), kw
