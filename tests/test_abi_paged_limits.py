"""CPU: further refusals of the paged-cache entry points, by the C ABI (the pointers
are never followed) and by the Python binding."""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn
from gated_delta_rule_106_b200 import _build

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def test_plan_capacity_is_refused_before_outputs_are_made(lib):
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_page_plan(i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16,
                          token_capacity=(1 << 30) + 1)
    assert e.value.status == INVALID
