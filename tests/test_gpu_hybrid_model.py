"""The hybrid model of the examples: prompts in chunks of any size and prompts
fed whole, and decoded tokens against the same tokens fed as a prompt."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A layer rounds about ten values to bf16 on a row's way (norm, projection, rotation, weights,
# output, projection, sum), each off by at most 2^-8 and 2^-8 / sqrt(3) in the mean; four layers, the
# head, and two runs that round apart: sqrt(2 * 41) * 2^-8 / sqrt(3) = 0.0204, and half as much again
# for what the layers pass on.
TOL = 0.03


def example():
    spec = importlib.util.spec_from_file_location("hybrid_model", os.path.join(ROOT, "examples", "hybrid_model.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return ((a - b).float().norm() / b.float().norm()).item()


def draw(lens):
    gen = torch.Generator().manual_seed(2)
    return [torch.randint(0, 1024, (n,), generator=gen).to("cuda") for n in lens]


@pytest.mark.parametrize("chunk", [64, 100, 256])
@pytest.mark.parametrize("kw", [dict(), dict(window=150, softcap=20.0)])
def test_chunks_equal_whole(chunk, kw):
    m = example()
    prompts = draw([700, 130, 1, 256])
    a = m.generate(prompts, chunk, 0, **kw)[0]
    b = m.generate(prompts, 700, 0, **kw)[0]
    assert torch.isfinite(a).all() and rel(a, b) <= TOL


def test_decoded_tokens_equal_the_same_tokens_fed():
    m = example()
    prompts = draw([126, 40, 1])
    _, out, last, _ = m.generate(prompts, 64, 6)
    fed = [torch.cat([t, o]) for t, o in zip(prompts, out)]
    again = m.generate(fed, 200, 0)[0]
    assert rel(last, again) <= TOL
