"""Automatic differentiation of ``rope``: gradients against the formula and against
differences, of views, of one output alone, broadcast ones, twice; what is refused."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def close(got, want, x, dtype, rot, tab, what=""):
    a, u = au.rotation_bounds(x, dtype, rot, tab)
    err = np.abs(au.f64(got) - want)
    assert (err <= a * (1 + u) + u * np.abs(want) + au.TINY[dtype]).all(), what


def setup(T, Hq, Hk, D, rot, dtype, seed=0):
    qkv = au.queries(T, Hq + 2 * Hk, D, dtype, seed, DEV).requires_grad_()
    tab = lib().rope_table(40, rot)
    pos = torch.arange(T, device=DEV) * 3 % 40
    return qkv, tab, pos


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("interleaved,transposed", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32), (80, 20)])
def test_gradient_of_a_fused_projection(D, rot, dtype, interleaved, transposed):
    T, Hq, Hk = 9, 4, 2
    qkv, tab, pos = setup(T, Hq, Hk, D, rot, dtype)
    q, k, v = qkv.split([Hq, Hk, Hk], dim=1)
    qo, ko = lib().rope(q, k, tab, pos, interleaved, transposed)
    assert qo.requires_grad and ko.requires_grad
    wq, wk = au.queries(T, Hq, D, dtype, 1, DEV), au.queries(T, Hk, D, dtype, 2, DEV)
    torch.autograd.backward([qo, ko], [wq, wk])
    want = [oatt.rotate(au.f64(w), au.f64(tab), pos.tolist(), interleaved, not transposed) for w in (wq, wk)]
    close(qkv.grad[:, :Hq], want[0], au.f64(wq), dtype, rot, au.f64(tab), "q")
    close(qkv.grad[:, Hq:Hq + Hk], want[1], au.f64(wk), dtype, rot, au.f64(tab), "k")
    assert (qkv.grad[:, Hq + Hk:] == 0).all()
    # the same values as without a gradient
    with torch.no_grad():
        a, b = lib().rope(q, k, tab, pos, interleaved, transposed)
    assert not a.requires_grad and torch.equal(a, qo) and torch.equal(b, ko)


def test_one_output_alone_and_no_keys():
    qkv, tab, pos = setup(5, 3, 2, 64, 64, FP)
    q, k, _ = qkv.split([3, 2, 2], dim=1)
    _, ko = lib().rope(q, k, tab, pos)
    w = au.queries(5, 2, 64, FP, 3, DEV)
    ko.backward(w)
    assert (qkv.grad[:, :3] == 0).all()
    close(qkv.grad[:, 3:5], oatt.rotate(au.f64(w), au.f64(tab), pos.tolist(), False, True), au.f64(w), FP, 64, au.f64(tab))
    qkv.grad = None
    qo, none = lib().rope(q, None, tab, pos)
    assert none is None
    qo.backward(torch.ones_like(qo))
    ones = np.ones((5, 3, 64))
    close(qkv.grad[:, :3], oatt.rotate(ones, au.f64(tab), pos.tolist(), False, True), ones, FP, 64, au.f64(tab))
    # keys alone require a gradient
    q0, k0 = q.detach(), k.detach().clone().requires_grad_()
    qo, ko = lib().rope(q0, k0, tab, pos)
    (qo.sum() + ko.sum()).backward()
    close(k0.grad, oatt.rotate(ones[:, :2], au.f64(tab), pos.tolist(), False, True), ones[:, :2], FP, 64, au.f64(tab))


def test_broadcast_gradients():
    """A sum's gradient is one value with strides of zero; a head's mean is one row for all heads."""
    qkv, tab, pos = setup(6, 2, 2, 64, 32, FP)
    q, k, _ = qkv.split([2, 2, 2], dim=1)
    qo, ko = lib().rope(q, k, tab, pos)
    w = au.queries(6, 1, 64, FP, 4, DEV)[:, 0]
    (qo.sum() + (ko.mean(dim=1) * w).sum()).backward()
    ones = np.ones((6, 2, 64))
    close(qkv.grad[:, :2], oatt.rotate(ones, au.f64(tab), pos.tolist(), False, True), ones, FP, 32, au.f64(tab))
    half = np.repeat(au.f64(w)[:, None] / 2, 2, axis=1)
    close(qkv.grad[:, 2:4], oatt.rotate(half, au.f64(tab), pos.tolist(), False, True), half, FP, 32, au.f64(tab))


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """The map is linear, so a difference over a step of 1 is the derivative; both sides' outputs round by 2^-22
    of a pair's values, and w weighs them."""
    T, D, rot = 2, 8, 6
    x = au.queries(T, 1, D, FP, 5, DEV).requires_grad_()
    tab, pos = lib().rope_table(40, rot), torch.tensor([7, 31], device=DEV)
    w = au.queries(T, 1, D, FP, 6, DEV)

    def f(t):
        return float((au.f64(lib().rope(t, None, tab, pos, interleaved)[0]) * au.f64(w)).sum())

    lib().rope(x, None, tab, pos, interleaved)[0].backward(w)
    with torch.no_grad():
        at = f(x)
        top = float(x.abs().max()) + 1
        lim = 2 * float(w.abs().sum()) * 2 * top * 2.0 ** -22 + float(w.abs().max()) * 2.0 ** -21
        for t in range(T):
            for d in range(D):
                y = x.detach().clone()
                y[t, 0, d] += 1
                step = float(y[t, 0, d].double() - x[t, 0, d].double())
                assert abs((f(y) - at) / step - float(x.grad[t, 0, d])) <= lim * 1.01


def test_twice():
    qkv, tab, pos = setup(4, 2, 1, 64, 64, FP)
    q = qkv[:, :2]
    qo, _ = lib().rope(q, None, tab, pos)
    (g,) = torch.autograd.grad((qo ** 2).sum(), q, create_graph=True)
    # sum of squares is kept by the rotation: its gradient is 2 q, and the gradient of that 2
    close(g, 2 * au.f64(q), 2 * au.f64(q), FP, 64, np.concatenate([au.f64(tab)] * 2))
    (h,) = torch.autograd.grad(g.sum(), q)
    two = np.full(h.shape, 2.0)
    close(h, two, two, FP, 64, np.concatenate([au.f64(tab)] * 2))


def test_refusals():
    qkv, tab, pos = setup(4, 2, 1, 64, 64, FP)
    q = qkv[:, :2]
    with pytest.raises(RuntimeError, match="automatic differentiation"):
        lib().rope(q, None, tab, pos, q_out=torch.empty(4, 2, 64, device=DEV))
    with pytest.raises(RuntimeError, match="table"):
        lib().rope(q.detach(), None, tab.clone().requires_grad_(), pos)
    with torch.no_grad():
        out = torch.empty(4, 2, 64, device=DEV)
        assert lib().rope(q, None, tab, pos, q_out=out)[0] is out
