"""The attention calls' workspace: 256-byte aligned, as the prefill's beside them."""

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn
from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _AttentionC, _CacheC, _RowsC

EWORKSPACE = -4
FAKE = 1 << 20  # an address the calls below never reach


@pytest.mark.parametrize("off", [1, 4, 8, 16, 64, 128, 255])
def test_unaligned_addresses_are_refused(off):
    lib = _lib.load()
    d = _AttentionC(4, 2, 64, 0, 0.0, 0.0, 0, 1)
    c = _CacheC(FAKE, FAKE, 2 * 16 * 64, 2 * 64, 64, 16, 2, FAKE, FAKE, FAKE)
    q, out = _RowsC(FAKE, 4 * 64, 64), _RowsC(2 * FAKE, 4 * 64, 64)
    for rc in (lib.gdn_attention_prefill_paged(d, q, FAKE, 2, c, out, None, FAKE + off, 1 << 40, None),
               lib.gdn_attention_decode_paged(d, q, c, out, None, FAKE + off, 1 << 40, None)):
        assert rc == EWORKSPACE
        assert "256-byte aligned" in lib.gdn_last_error().decode()


@pytest.mark.gpu
def test_a_callers_workspace():
    dev, bf = "cuda", torch.bfloat16
    c = au.batch([50, 700], 16, 2, 64, bf, 0, dev)
    q, cu = au.queries(2, 8, 64, bf, 1, dev), au.i32([0, 1, 2], dev)
    n = gdn.attention_workspace_size(2, 2, 8, 2, 64)
    ws = torch.empty(n + 512, dtype=torch.uint8, device=dev)
    for call in (lambda w: gdn.attention_decode_paged(q, **c, workspace=w),
                 lambda w: gdn.attention_prefill_paged(q, cu, **c, workspace=w)):
        ref = call(None)
        assert torch.equal(call(ws[256:]), ref) and torch.equal(call(ws[:n]), ref)
        for bad in (ws[8:], ws[16:], ws[128:]):
            with pytest.raises(gdn.GDNError, match="aligned"):
                call(bad)
        with pytest.raises(ValueError):
            call(ws[:n - 1])
