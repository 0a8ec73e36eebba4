"""Shared attention on the GPU with as many sequences and groups as there may be, for every cache type and the largest heads: the
launches with the most LDS."""
import pytest

import rank_adapter_gemm_build_amd as rx
from test_gpu_shared_attention import call, near_paged, shared_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("groups,news,hq", [(4096, 1, 1), (4096, 17, 2), (1024, 1, 1), (1024, 40, 1)])
def test_most_sequences_and_groups(groups, news, hq, dim, cache):
    S = rx.LORA_MAX_SEQS
    per = S // groups
    case = shared_case(groups + dim, [(16 + i % 5, [news + (i + j) % 7 for j in range(per)]) for i in range(groups)], news, hq, 1, dim, cache)
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, hq, 1, dim, scales)
    near_paged(case, hq, 1, dim, scales, out, lse, f"{S} sequences in {groups} groups {dim} {cache}")
