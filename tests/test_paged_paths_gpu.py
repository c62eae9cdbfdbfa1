"""Calls of the paged cache that the sizes of the other tests pass by: counts far past the capacity."""
import numpy as np
import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base

pytestmark = pytest.mark.gpu
gen = base.gen


@pytest.mark.parametrize("B,cu", [(450, None), (2, None), (3, [0, 2, 2, 5])], ids=["many rows", "few rows", "several tokens"])
def test_counts_past_the_capacity_mean_full_rows(B, cu):
    """A count beyond the capacity, the largest int32 too, is a full row, and its count is the capacity afterwards."""
    a = ref.make_cache(B, 1, 64, 8, 40, seed=1)
    base.fill_random(a, [[40 + (b % 3)] for b in range(B)], seed=2)
    a["count"][::2] = 2 ** 31 - 1
    base.check_append(a, cu, 8, 2, seed=3)
    touched = [b for b in range(B) if cu is None or cu[b + 1] > cu[b]]
    assert a["count"].cpu()[touched].eq(40).all()
