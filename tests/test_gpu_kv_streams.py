"""Objects of the paged-cache operators made while their device is busy and used on another stream at once."""
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from test_gpu_kv import ints

pytestmark = pytest.mark.gpu


def test_a_plan_is_ready_for_any_stream():
    """The vectors' first fill is over before a step on another stream writes them."""
    past, new = ints([5, 16, 0]), ints([2, 1, 3])
    table, ring, cursor = ints([0, -1, -1] * 3).view(3, 3), ints([7, 6, 5, 4, 3, 2, 1, 0]), ints([0, 4, 0, 0])
    s = torch.cuda.Stream()
    busy = torch.ones(1 << 27, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):
        busy.mul_(1.0)                    # some 20 ms on the current stream
    plan = rx.PagePlan(0, 3, 6)
    rx.page_plan(plan, past, new, 6, ring, cursor, table, 16, stream=s)
    torch.cuda.synchronize()
    assert plan.seq_lens.tolist() == [7, 17, 3] and plan.query_start.tolist() == [0, 2, 3, 6]
    assert plan.positions.tolist() == [5, 6, 16, 0, 1, 2]
    assert plan.slots.tolist() == [5, 6, 7 * 16, 6 * 16, 6 * 16 + 1, 6 * 16 + 2]
    assert plan.meta.tolist() == [6, 2, 0, 0, 0, 2, 0, 0]
