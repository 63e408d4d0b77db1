"""The build refuses kernels that move vector registers between the two register files, but for the listed ones
up to their number (CPU: the compiler's remarks are made up)."""

import types

import pytest

from paged_recurrent_state_amd import build

LISTED = sorted(build.MOVED)[0]


def compile_with(monkeypatch, tmp_path, name, regs, scratch):
    remarks = "".join(f"a.hip:1:1: remark: {what}: {x} [-Rpass-analysis=kernel-resource-usage]\n" for what, x in (
        ("Function Name", name), ("    ScratchSize [bytes/lane]", scratch), ("    VGPRs Spill", regs)))

    def run(cmd, **kw):
        (tmp_path / "a.o").write_text("")
        return types.SimpleNamespace(returncode=0, stderr=remarks)

    monkeypatch.setattr(build.subprocess, "run", run)
    try:
        return build._compile("a.hip", str(tmp_path), str(tmp_path))
    finally:
        monkeypatch.undo()


@pytest.mark.parametrize("name,regs,scratch", [("kernel", 1, 0), ("kernel", 0, 4), ("kernel", 1, 4), (LISTED, 2, 0), (LISTED, 1, 4)])
def test_refused(monkeypatch, tmp_path, name, regs, scratch):
    with pytest.raises(RuntimeError, match="spill"):
        compile_with(monkeypatch, tmp_path, name, regs, scratch)
    assert not (tmp_path / "a.o").exists()


@pytest.mark.parametrize("name,regs", [("kernel", 0), (LISTED, 0), (LISTED, build.MOVED[LISTED])])
def test_taken(monkeypatch, tmp_path, name, regs):
    assert compile_with(monkeypatch, tmp_path, name, regs, 0) == str(tmp_path / "a.o")


def test_the_listed_ones_are_kernels_of_the_library():
    with open(build.LIB, "rb") as f:
        built = f.read()
    assert build.MOVED and all(name.encode() in built and regs == 1 for name, regs in build.MOVED.items())
