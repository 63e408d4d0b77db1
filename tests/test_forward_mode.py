"""Forward-mode differentiation: the rotation and the norm before it have no tangents, so dual tensors are
refused, not taken for ordinary ones (CPU: refused before anything else is asked)."""

import pytest
import torch
from torch.autograd import forward_ad

import paged_recurrent_state_amd as gdn


def inputs(device="cpu"):
    names = dict(q=(3, 4, 64), k=(3, 2, 64), q_weight=(64,), k_weight=(64,), table=(8, 32))
    x = {n: torch.ones(s, device=device) for n, s in names.items()}
    return x, torch.arange(3, device=device)


def calls(x, pos):
    rows = (x["q"], x["k"], x["q_weight"], x["k_weight"], x["table"], pos)
    return {"rope": lambda: gdn.rope(x["q"], x["k"], x["table"], pos),
            "rope_backward": lambda: gdn.rope_backward(x["q"], x["k"], x["table"], pos),
            "norm_rope": lambda: gdn.norm_rope(*rows),
            "norm_rope_backward": lambda: gdn.norm_rope_backward(x["q"], x["k"], *rows)}


TAKES = [(call, dual) for call in ("rope", "rope_backward", "norm_rope", "norm_rope_backward")
         for dual in ("q", "k", "q_weight", "k_weight", "table") if "norm" in call or "weight" not in dual]


@pytest.mark.parametrize("call,dual", TAKES)
@pytest.mark.parametrize("leaf", [False, True])
def test_dual_tensors_are_refused(dual, call, leaf):
    x, pos = inputs()
    with forward_ad.dual_level():
        x[dual] = forward_ad.make_dual(x[dual].requires_grad_(leaf), torch.ones_like(x[dual]))
        with pytest.raises(RuntimeError, match="forward-mode"):
            calls(x, pos)[call]()
        with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
            calls(x, pos)[call]()


@pytest.mark.parametrize("name", ["q_out", "k_out"])
def test_dual_outputs_are_refused(name):
    x, pos = inputs()
    with forward_ad.dual_level():
        out = {name: forward_ad.make_dual(torch.ones_like(x[name[0]]), torch.ones_like(x[name[0]]))}
        for call in (lambda: gdn.rope(x["q"], x["k"], x["table"], pos, **out),
                     lambda: gdn.norm_rope(x["q"], x["k"], x["q_weight"], x["k_weight"], x["table"], pos, **out)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()


def test_ordinary_tensors_at_a_dual_level_are_not():
    x, pos = inputs()
    with forward_ad.dual_level():
        for call in calls(x, pos).values():
            with pytest.raises(ValueError, match="no CPU path"):
                call()


@pytest.mark.gpu
def test_at_a_dual_level_the_results_are_the_same():
    x, pos = inputs("cuda")
    want = {n: f() for n, f in calls(x, pos).items()}
    with forward_ad.dual_level():
        for n, f in calls(x, pos).items():
            assert all(torch.equal(a, b) for a, b in zip(f(), want[n]))
        x["k"] = forward_ad.make_dual(x["k"], torch.ones_like(x["k"]))
        for f in calls(x, pos).values():
            with pytest.raises(RuntimeError, match="forward-mode"):
                f()
