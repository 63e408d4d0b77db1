"""The hybrid example with normed heads, an 8-bit cache and first tokens beside a window:
prompts in chunks and fed whole, decoded tokens against the same tokens fed, and a
training step through the norms."""

import pytest
import torch

from test_gpu_hybrid_model import TOL, draw, example, rel

pytestmark = pytest.mark.gpu

# With an 8-bit cache a chunk's end inside a block of 16 tokens rounds earlier rows' codes once more where the
# block's scale grows (exact but for codes that become subnormal), and two runs' keys, which differ by bf16
# roundings (2^-8), fall on other codes: a code that flips is off by 2^-3 of its value at most.  A difference of d in a
# key flips a code with the probability d / (2^-3 value), so that the mean square of what codes differ by is
# 2^-3 times d's mean size, 2^-3 * 2^-8 = 2^-11, a relative error of 0.022 in every key and value, of which
# attention over n keys keeps 1/sqrt(n) in the mean (the first tokens, which see one, all of it), in one layer
# of four: well under a further 0.03.
TOL8 = 2 * TOL

OPTIONS = [(dict(norms=True), TOL), (dict(window=150, sinks=5), TOL), (dict(cache8=True), TOL8),
           (dict(norms=True, cache8=True, window=100, sinks=20, softcap=20.0), TOL8)]


@pytest.mark.parametrize("kw,tol", OPTIONS)
@pytest.mark.parametrize("chunk", [64, 100])
def test_chunks_equal_whole(chunk, kw, tol):
    m = example()
    prompts = draw([700, 130, 1, 256])
    a = m.generate(prompts, chunk, 0, **kw)[0]
    b = m.generate(prompts, 700, 0, **kw)[0]
    assert torch.isfinite(a).all() and rel(a, b) <= tol


@pytest.mark.parametrize("kw,tol", OPTIONS)
def test_decoded_tokens_equal_the_same_tokens_fed(kw, tol):
    m = example()
    prompts = draw([126, 40, 1])
    _, out, last, _ = m.generate(prompts, 64, 6, **kw)
    fed = [torch.cat([t, o]) for t, o in zip(prompts, out)]
    again = m.generate(fed, 200, 0, **kw)[0]
    assert rel(last, again) <= tol


def test_command(capsys):
    example().main(["--prompts", "70", "9", "--chunk", "32", "--tokens", "2", "--norms", "--cache8", "--window", "40", "--sinks", "4"])
    assert "2 tokens decoded" in capsys.readouterr().out


def test_a_training_step_through_the_norms():
    """The projection, the norms with the rotation and a loss: every gradient against the same step in torch's own
    operations in 64 bits."""
    import paged_recurrent_state_amd as gdn
    T, H, Hk, D, hidden = 24, 4, 2, 64, 96
    gen = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x, target = randn(T, hidden), randn(T, H + Hk, D)
    w = (randn(hidden, (H + Hk) * D) * hidden ** -0.5).requires_grad_()
    wq, wk = (1 + 0.1 * randn(D)).requires_grad_(), (1 + 0.1 * randn(D)).requires_grad_()
    table, pos = gdn.rope_table(64, D), torch.arange(T, device="cuda")
    q, k = (x @ w).view(T, H + Hk, D).split([H, Hk], dim=1)
    q, k = gdn.norm_rope(q, k, wq, wk, table, pos)
    (torch.cat([q, k], dim=1) * target).sum().backward()
    got = [t.grad.double() for t in (w, wq, wk)]

    w64, wq64, wk64 = (t.detach().double().requires_grad_() for t in (w, wq, wk))
    y = (x.double() @ w64).view(T, H + Hk, D)
    y = y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * torch.cat([wq64.expand(H, D), wk64.expand(Hk, D)])
    c, s = table.double()[pos].split(D // 2, dim=1)
    a, b = y[..., :D // 2], y[..., D // 2:]
    y = torch.cat([a * c[:, None] - b * s[:, None], b * c[:, None] + a * s[:, None]], dim=-1)
    (y * target.double()).sum().backward()
    for g, t in zip(got, (w64, wq64, wk64)):
        # fp32 throughout: sums of at most 24 * 4 rows and a product over 96 or 24 values, 2^-24 a step
        assert (g - t.grad).norm() <= 2.0 ** -16 * t.grad.norm()
