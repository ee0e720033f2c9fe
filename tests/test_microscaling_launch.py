"""What the launchers of the microscaled kernels refuse by themselves, whatever chose them.  Their host code alone is compiled
and run here, with no device to launch on; needs no GPU."""
import os
import subprocess

import pytest

from post_weight_quantization_group_amd import build

PROGRAM = """
#include <stdio.h>
#include "mxlinear.hip"
hipError_t cqk::launch_mx_rows(const MxRowsArgs&, bool, hipStream_t) { return hipErrorNotSupported; }
int main(int, char** v) {
    cqk::MxLinearArgs a{};
    a.M = 4096, a.out = 4096, a.in = atoi(v[1]);
    printf("%d %d %d", cqk::many<cqk::MXFP4, false, 256, 256, 2>(a, nullptr) == hipErrorInvalidValue,
           cqk::many<cqk::MXFP4, true, 128, 128, 3>(a, nullptr) == hipErrorInvalidValue,
           cqk::many<cqk::MXFP8, false, 128, 128, 2>(a, nullptr) == hipErrorInvalidValue);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("launch")
    (at / "program.hip").write_text(PROGRAM)
    # the kernels themselves are not compiled: what would hold them stays undefined
    subprocess.run([build._hipcc(), "-x", "hip", f"--offload-arch={build.ARCH}", "--offload-host-only", *build.COMMON, "-O1",
                    "-Wl,--unresolved-symbols=ignore-all", str(at / "program.hip"), "-o", str(at / "program")],
                   check=True, capture_output=True, timeout=300)
    return at / "program"


@pytest.mark.parametrize("k,refused", [(64, "1 1 1"), (128, "1 0 0"), (160, "1 1 1"), (384, "1 0 0")])
def test_linear_over_many_rows_takes_whole_steps_of_k_only(program, k, refused):
    """in < a step would leave no step, and loads in front of x and W; a remainder would be left out of the sums."""
    run = subprocess.run([str(program), str(k)], capture_output=True, text=True, timeout=60,
                         env={**os.environ, "HIP_VISIBLE_DEVICES": "-1", "ROCR_VISIBLE_DEVICES": "-1"})
    assert run.returncode == 0 and run.stdout == refused
