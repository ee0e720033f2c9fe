"""The serving kernels' instructions as the build compiles them: no register goes to memory (scratch), and no access
is generic (flat), whose address could be anywhere.  Compiled here from the sources; needs no GPU."""
import os
import re
import subprocess

import pytest

from post_weight_quantization_group_amd import build


@pytest.mark.parametrize("name", ["attention", "linear", "kvcache"])
def test_neither_spills_nor_generic_accesses(name, tmp_path):
    out = tmp_path / "kernels.s"
    cmd = [build._hipcc(), "-x", "hip", f"--offload-arch={build.ARCH}", *build.COMMON, "--cuda-device-only", "-S",
           os.path.join(build.CSRC, name + ".hip"), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=600)
    text = out.read_text()
    assert re.search(r"^\s+global_load_", text, re.M)
    assert not re.findall(r"^\s+(?:flat|scratch)_(?:load|store|atomic)\w*.*$", text, re.M)
    assert set(re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)) == {"0"}
    assert set(re.findall(r"\.vgpr_spill_count:\s*(\d+)", text)) == {"0"}
