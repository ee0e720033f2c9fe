"""The microscaled kernels' instructions as the build compiles them: no register goes to memory (scratch), and no access
is generic (flat), whose address could be anywhere.  Compiled here from the sources; needs no GPU."""
import pytest

from test_serving_isa import test_neither_spills_nor_generic_accesses as _check


@pytest.mark.parametrize("name", ["attention_mx", "mx", "mxlinear"])
def test_neither_spills_nor_generic_accesses_mx(name, tmp_path):
    _check(name, tmp_path)
