"""Results while another stream fills the load and store units: reads of a ring's slot stay in front of its next copy."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PagedCase
from query_aware_sparse_quest_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def repeats(call):
    """The same bits alone and beside transposed copies, whose stores take a sector each."""
    noise = torch.randn((4096, 4096), device=DEV)
    sink, side = torch.empty_like(noise), torch.cuda.Stream()
    first = call()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            for _ in range(4):
                sink.copy_(noise.t())
        got = [call() for _ in range(10)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, x) for x in got)
    assert binding.sv_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [1, 16, 90])
def test_window_attention_repeats_exactly_beside_scattered_stores(size, fp8):
    case = PagedCase([1500 + 37 * i for i in range(24)], 2, fp8=fp8)
    rows, cache, table = 24 * size, case.cache(), case.table.to(DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    lens, starts = ints(case.lens), None if size == 1 else ints([size * b for b in range(25)])
    q = torch.randn((rows, 16, DIM), device=DEV).bfloat16()
    ws = torch.empty(binding.sv_window_attention_workspace_size(24, 16, 2, rows), dtype=torch.uint8, device=DEV)

    def call():
        out, lse = torch.empty_like(q), torch.empty((rows, 16), device=DEV)
        binding.sv_window_attention(cache, q, table, lens, 1000, 5, out, lse, ws, q_start=starts)
        return torch.cat([out.float().flatten(), lse.flatten()])
    repeats(call)
