"""The example's command: no tokens to decode, and arguments it cannot run."""

import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_model", os.path.join(ROOT, "examples", "hybrid_model.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("argv", [["--prompts", "5", "0"], ["--prompts", "-1"], ["--chunk", "0"], ["--tokens", "-1"]])
def test_arguments_that_cannot_run(example, argv, capsys):
    with pytest.raises(SystemExit) as e:
        example.main(argv)
    assert e.value.code == 2 and "token" in capsys.readouterr().err


def test_generate_refuses_empty_prompts(example):
    some = torch.zeros(3, dtype=torch.int64)
    for prompts, chunk, tokens in (([], 4, 1), ([some, some[:0]], 4, 1), ([some], 0, 1), ([some], 4, -1)):
        with pytest.raises(ValueError):
            example.generate(prompts, chunk, tokens, device="cpu")


@pytest.mark.gpu
def test_no_tokens_to_decode(example, capsys):
    example.main(["--prompts", "40", "1", "--chunk", "16", "--tokens", "0"])
    out = capsys.readouterr().out
    assert "logits within" in out and "decoded" not in out


@pytest.mark.gpu
def test_some_tokens(example, capsys):
    example.main(["--prompts", "40", "1", "--chunk", "16", "--tokens", "2"])
    lines = capsys.readouterr().out.splitlines()
    assert "2 tokens decoded" in lines[1] and [len(x.split()) for x in lines[2:]] == [2, 2]
