"""sv_pages_* where lists and tables hold what they should not, and called right before the calls that read what
they write."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PAGE, attend, check, window_seen
from query_aware_sparse_quest_gb300 import binding
from test_gpu_pages import Device, Model, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("first", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30, 7])
@pytest.mark.parametrize("end", [2 ** 31 - 1, 9, -2 ** 31])
def test_freeing_pages_behind_a_row_does_nothing(first, end):
    d = Device(Model(40, 3, 12))
    d.reserve([0, 1], [100, 190])
    d.free([0, 1, 0], [first, max(first, 12), first], [end] * 3)
    d.same()
