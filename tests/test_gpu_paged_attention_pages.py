"""GPU: block tables whose entries lie outside the pool, at the ends of 32 bits among them (cq_paged_attention)."""
import pytest

import post_weight_quantization_group_amd as cq
from parity import say
from serving import Paged, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [-1, -2, -(1 << 31), -(1 << 31) + 1, (1 << 31) - 1])
@pytest.mark.parametrize("at", [0, 4, 18])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 90)], [(100, 300), (2, 90)]])
def test_entries_outside_the_pool_are_masked(lens, at, page):
    """Also where nothing else marks the key as missing: few rows and many, the first, a middle and the last page."""
    say("pages outside", lens, at, page)
    p = Paged(lens, 4, 2, 128, 16, "bf16")
    p.table_np[0, at] = page
    p.table = i32(p.table_np)
    p.check(cq)
