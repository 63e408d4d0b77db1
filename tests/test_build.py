"""The build refuses kernels that keep vector registers in memory (CPU: compiles two small sources)."""

import pytest

from paged_recurrent_state_amd import build

# 120 values of a thread live over a barrier, at 1,024 threads a workgroup (64 registers each) or 256
SOURCE = """
#include <hip/hip_runtime.h>
extern "C" __global__ __launch_bounds__(%d) void wide(const float* x, float* y) {
  float v[120];
#pragma unroll
  for (int i = 0; i < 120; ++i) v[i] = x[i * 1024 + threadIdx.x];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 120; ++i) y[((i * 7) %% 120) * 1024 + threadIdx.x] = v[i] * v[(i * 31 + 5) %% 120];
}
"""


def test_a_kernel_that_spills_is_refused(tmp_path):
    (tmp_path / "wide.hip").write_text(SOURCE % 1024)
    with pytest.raises(RuntimeError, match="spill.*wide"):
        build._compile("wide.hip", str(tmp_path), str(tmp_path))
    assert not (tmp_path / "wide.o").exists()


def test_one_that_fits_is_not(tmp_path):
    (tmp_path / "wide.hip").write_text(SOURCE % 256)
    obj = build._compile("wide.hip", str(tmp_path), str(tmp_path))
    assert obj == str(tmp_path / "wide.o") and (tmp_path / "wide.o").exists()


def test_remarks():
    def remark(name, regs, scratch):
        at = "csrc/a.hip:42:1: remark: "
        return (f"{at}Function Name: {name} [-Rpass-analysis=kernel-resource-usage]\n   42 |   int64_t n) {{\n      | ^\n"
                f"{at}    ScratchSize [bytes/lane]: {scratch} [-Rpass-analysis=kernel-resource-usage]\n"
                f"{at}    SGPRs Spill: 7 [-Rpass-analysis=kernel-resource-usage]\n"
                f"{at}    VGPRs Spill: {regs} [-Rpass-analysis=kernel-resource-usage]\n")

    assert build.spills(remark("a", 0, 0) + remark("b", 2, 8) + remark("c", 1, 0) + "warning: VGPRs\n") == {
        "b": (2, 8), "c": (1, 0)}
    assert build.spills("") == {}
