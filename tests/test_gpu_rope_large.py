"""Rotary rows of more bytes than the caches hold, whose stores pass them: every
value against the same rows rotated a part at a time."""

import pytest
import torch

import attention_util as au

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,interleaved", [(torch.bfloat16, False), (torch.float16, True), (torch.float32, False)])
def test_large_equals_its_parts(dtype, interleaved):
    import paged_recurrent_state_amd as m
    T, Hq, Hk, D = 9001, 16, 4, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(T, Hq, D, generator=gen, device=DEV).to(dtype)
    k = torch.randn(T, Hk, D, generator=gen, device=DEV).to(dtype)
    assert T * (Hq + Hk) * D * q.element_size() > 32 << 20
    tab = m.rope_table(T, 64)
    pos = torch.arange(T, device=DEV)
    qo, ko = m.rope(q, k, tab, pos, interleaved=interleaved)
    for lo in range(0, T, 1000):
        a, b = m.rope(q[lo:lo + 1000], k[lo:lo + 1000], tab, pos[lo:lo + 1000], interleaved=interleaved)
        assert torch.equal(a, qo[lo:lo + 1000]) and torch.equal(b, ko[lo:lo + 1000])


def test_large_append_equals_its_parts():
    import paged_recurrent_state_amd as m
    lens = [4000, 5001]
    T, Hq, Hk, D, page = sum(lens), 8, 4, 256, 64
    q, k, v = (au.queries(T, h, D, torch.bfloat16, s, DEV) for h, s in ((Hq, 1), (Hk, 2), (Hk, 3)))
    tab = m.rope_table(max(lens), 64)
    pages = [-(-n // page) for n in lens]
    idx = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(4)).to(torch.int32).to(DEV)

    def table(ns):
        ps = [-(-n // page) for n in ns]
        ptr = au.i32([0, pages[0], sum(pages)], DEV)
        assert ps == pages
        return idx, ptr, page, au.i32([n - (p - 1) * page for n, p in zip(ns, ps)], DEV)

    one = torch.zeros(2, sum(pages), page, Hk, D, dtype=torch.bfloat16, device=DEV)
    two = torch.zeros_like(one)
    q1 = m.kv_append_paged(k, v, au.i32([0, lens[0], T], DEV), one[0], one[1], *table(lens), table=tab, q=q)
    # 600 tokens at a time, each time with the page table as it is then
    q2 = torch.empty_like(q1)
    starts = [0, lens[0]]
    for b, n in enumerate(lens):
        for lo in range(0, n, 600):
            hi = min(n, lo + 600)
            ptr = au.i32([0, -(-hi // page)], DEV)
            rows = slice(starts[b] + lo, starts[b] + hi)
            part = idx[(0 if b == 0 else pages[0]):][:-(-hi // page)].contiguous()
            lpl = au.i32([hi - (-(-hi // page) - 1) * page], DEV)
            q2[rows] = m.kv_append_paged(k[rows], v[rows], au.i32([0, hi - lo], DEV), two[0], two[1], part, ptr, page,
                                         lpl, table=tab, q=q[rows])
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(q1, q2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(80, 48), (48, 0), (64, 64)])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_every_piece_width_gives_the_same_bits(dtype, interleaved, D, rot, shift):
    """Rows that start 0, 1, 2 and 4 values after an aligned address take pieces of other widths
    (rows of 81 values: one pair at a time); the values are those of aligned rows, bit by bit, and
    nothing beside the rows is written."""
    import paged_recurrent_state_amd as m
    T, H, page = 21, 3, 8
    cu, pages = au.i32([0, T], DEV), -(-T // page)
    where = (torch.arange(pages, dtype=torch.int32, device=DEV), au.i32([0, pages], DEV), page,
             au.i32([T - (pages - 1) * page], DEV))
    tab = m.rope_table(T, rot) if rot else None
    k, v = (au.queries(T, H, D, dtype, s, DEV) for s in (8, 9))
    outs = []
    for at, row in ((0, D), (shift, D + (shift == 1))):
        def rows(n, x=None):
            flat = torch.full((n * row + at + 5,), 7.0, dtype=dtype, device=DEV)
            view = flat[at:at + n * row].view(-1, H, row)[..., :D]
            if x is not None:
                view.copy_(x)
            return flat, view
        slots = pages * page * H
        (fk, ck), (fv, cv) = rows(slots), rows(slots)
        (_, kk), (_, vv) = rows(T * H, k), rows(T * H, v)
        m.kv_append_paged(kk, vv, cu, ck.unflatten(0, (pages, page)),
                          cv.unflatten(0, (pages, page)), *where, table=tab, interleaved=interleaved)
        torch.cuda.synchronize()
        outs.append((ck[:T].clone(), cv[:T].clone()))
        for flat, view in ((fk, ck), (fv, cv)):
            assert (view[T:] == 7).all() and (flat[:at] == 7).all() and (flat[at + slots * row:] == 7).all()
            if row > D:
                assert (flat[at:at + slots * row].view(-1, row)[:, D:] == 7).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(outs[0][1], v)
