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


def test_as_many_slots_as_an_index_counts():
    """A refused request for 2^31 - 6 tokens, behind one of 5: its slots are -1, up to the list's last."""
    most = 2 ** 31 - 1
    d = Device(Model(40, 3, 12))
    d.reserve([0], [10])
    slots = torch.full((most,), -99, dtype=torch.int32, device=DEV)
    binding.sv_pages_reserve(d.table, d.lens, d.counts, ints([0, 1]), ints([5, most - 5]), slots, d.ws)
    torch.cuda.synchronize()
    assert slots[:5].tolist() == d.m.reserve([0], [5])
    assert (slots[5:2 ** 30] == -1).all() and (slots[2 ** 30:] == -1).all()
    d.same(0x8)
