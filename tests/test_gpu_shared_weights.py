"""Shared attention on the GPU where groups have many rows: weights that are exactly 0, and scales at the ends of their range."""
import pytest
import torch

import test_gpu_kv as base
from test_gpu_shared_attention import call, shared_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [-float("inf"), -1e4])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("members", [3, 40, 70])
def test_values_of_weight_0_have_no_effect(members, dim, low):
    """Common keys whose scores are minus infinity, or so low that the weight is 0 in fp32, with values that are large: the same bits
    as with values of 0.  (A part whose keys are all low has weights of 1 relative to its own maximum, so that the sum of 71
    such values has to be finite in fp32: 71 * 3e36 < 3.4e38.)"""
    case = shared_case(members, [(200, [5 + i % 30 for i in range(members)])], 1, 8, 2, dim, "bf16")
    q, k, v, table, *_ = case
    q.view(members, 8, dim)[:, :, 0] = 8.0
    got = []
    for value in (0.0, 1e35, -3e36):
        for token in list(range(0, 40)) + list(range(101, 131)) + [199]:
            page, at = int(table[0][token // 16]), token % 16
            k[page, at, :, 0] = low
            v[page, at] = value
        got.append(call(case, 8, 2, dim))
    assert got[0][0].isfinite().all() and got[0][0].abs().max() > 0.1
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-39, -1e-39, 1e-44, 2e-38])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("members", [3, 40])
def test_scales_near_0(members, dim, scale):
    """Products of queries and keys of up to some 1e37, which such scales take to less than 1 (0 to 0: every key counts alike)."""
    case = shared_case(members, [(150, [1 + i % 30 for i in range(members)])], 1, 8, 2, dim, "bf16")
    q, k, v, table, lens, starts, _, _ = case
    q *= 1e18
    k *= 1e17
    out, lse = call(case, 8, 2, dim, scale=scale)
    base.check_attend(q, k, v, table, lens, starts, 16, 8, 2, dim, out, lse, scale, 0, (1.0, 1.0), f"scale {scale} {members}x{dim}")
