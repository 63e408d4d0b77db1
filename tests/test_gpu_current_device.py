"""Every call runs on its tensors' device when another one is current: it is made current for the call (one GPU
suffices: the current device's number is made up, and the change of device recorded)."""

import pytest
import torch

import attention_util as au
import workloads

pytestmark = pytest.mark.gpu
DEV, BF = "cuda:0", torch.bfloat16


def calls():
    import paged_recurrent_state_amd as m
    c = au.batch([40, 9], 16, 2, 64, BF, 0, DEV)
    where = {n: c[n] for n in ("page_indices", "page_indptr", "page_size", "last_page_len")}
    sc = {n: torch.ones(c["k_cache"].shape[0], 1, 2, device=DEV) for n in ("k_scale", "v_scale")}
    coded = {**where, **sc, **{n: torch.zeros(c[n].shape, device=DEV).to(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")}}
    q, k, cu = au.queries(2, 4, 64, BF, 1, DEV), au.queries(2, 2, 64, BF, 2, DEV), au.i32([0, 1, 2], DEV)
    tab, pos = m.rope_table(64, 64, device=DEV), torch.arange(2, device=DEV)
    w = torch.ones(64, device=DEV)
    src = torch.zeros(64, device=DEV)
    yield "rope_table", lambda: m.rope_table(8, 64, device=DEV)
    yield "rope", lambda: m.rope(q, k, tab, pos)
    yield "rope_backward", lambda: m.rope_backward(q, k, tab, pos)
    yield "norm_rope", lambda: m.norm_rope(q, k, w, w, tab, pos)
    yield "norm_rope_backward", lambda: m.norm_rope_backward(q, k, q, k, w, w, tab, pos)
    yield "kv_append_paged", lambda: m.kv_append_paged(k, k, cu, **c)
    yield "kv_append_paged norms", lambda: m.kv_append_paged(k, k, cu, **c, k_norm=w)
    yield "kv_append_paged codes", lambda: m.kv_append_paged(k, k, cu, **coded)
    yield "kv_read_paged", lambda: m.kv_read_paged(cu, 2, **coded)
    for name, kv in (("", c), (" codes", coded)):
        for more in ({}, dict(window=5, sinks=2)):
            yield f"prefill{name} {more}", lambda kv=kv, more=more: m.attention_prefill_paged(q, cu, **kv, **more)
            yield f"decode{name} {more}", lambda kv=kv, more=more: m.attention_decode_paged(q, **kv, **more)
    yield "stream_copy", lambda: m.stream_copy(src.clone(), src)
    tables = (where["page_indices"], where["page_indptr"], where["last_page_len"])
    yield "prefill_slots", lambda: m.prefill_slots(cu, *tables, 64)
    yield "decode_slots", lambda: m.decode_slots(*tables)
    yield "check_paged", lambda: m.check_paged(*tables, 64, 10)
    yield "csr_to_block_table", lambda: m.csr_to_block_table(tables[1], tables[0], tables[2], 64, 4)
    yield "block_table_to_csr", lambda: m.block_table_to_csr(torch.zeros(2, 4, dtype=torch.int32, device=DEV), au.i32([3, 5], DEV), 64)
    for form, call in (("prefill", m.prefill_paged), ("prefill", m.prefill_paged_noalloc), ("decode", m.decode_paged)):
        d = workloads.config0()
        x = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in d[form].items()}
        args = [x[n] for n in ("q", "k", "v", "g", "beta")] + ([x["cu_seqlens"]] if form == "prefill" else [])
        args += [d["pool"].to(DEV), x["page_indices"], x["page_indptr"], 128, x["last_page_len"]]
        yield call.__name__, lambda call=call, args=args: call(*args)
        rows = args[:6] if form == "prefill" else args[:5]
        state = args[len(rows)]
        index = dict(state_indices=x["page_indices"][:len(x["last_page_len"])]) if form == "prefill" else dict(
            initial_state_indices=x["page_indices"][:len(x["last_page_len"])])
        yield form, lambda call=getattr(m, form), rows=rows, more=dict(initial_state=state, **index): call(*rows, **more)


def test_calls_change_to_their_tensors_device(monkeypatch):
    for name, call in calls():
        call()
        entered = []

        class device(torch.cuda.device):
            def __enter__(self):
                entered.append(self.idx)

            def __exit__(self, *error):
                return False

        with monkeypatch.context() as mp:
            mp.setattr(torch._C, "_cuda_getDevice", lambda: 1)
            mp.setattr(torch.cuda, "device", device)
            call()
        assert entered == [0], name
        entered.clear()
        with monkeypatch.context() as mp:
            mp.setattr(torch.cuda, "device", device)
            call()
        assert not entered, name
    torch.cuda.synchronize()
