"""Decode attention over rows that are dealt out in shares: many more rows than a CTA holds the sizes of, and the
weights, which the attention adds for some rows and the second kernel for the others."""
import math

import numpy as np
import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base
from kernel_launches import launches
from test_paged_limits_gpu import word  # noqa: F401

pytestmark = pytest.mark.gpu
gen = base.gen


def decode_launches(a, q, accumulate):
    cache = kv.PagedCache(**a)
    B, Hq, d = q.shape
    out, lse = torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, device="cuda")
    ws = torch.empty(max(256, kv.paged_decode_workspace_bytes(cache, Hq, accumulate)), dtype=torch.uint8, device="cuda")
    return launches(lambda s: kv.paged_decode_attention(q, cache, accumulate=accumulate, out=out, lse=lse, workspace=ws, stream=s))


@pytest.mark.parametrize("dtype,G", [("bf16", 2), ("e4m3", 12)])
def test_shares_of_more_rows_than_are_held(dtype, G):
    """More than 1,024 rows, most of them short or empty, each CTA a share of the line."""
    B, H, cap = 270, 4, 1100
    rng = np.random.default_rng(3)
    counts = np.where(rng.random((B, H)) < 0.05, cap, rng.integers(-1, 5, (B, H))).tolist()
    a = ref.make_cache(B, H, 64, 64, cap, dtype, seed=1)
    base.fill_random(a, counts, seed=2)
    q = torch.randn(B, G * H, 64, generator=gen(1)).to(torch.bfloat16).cuda()
    for accumulate in (False, True):
        got = decode_launches(a, q, accumulate)
        assert ["paged_decode_kernel" in got[0][0], "paged_join_kernel" in got[1][0], len(got)] == [True, True, 2]
        assert got[0][1] < B * H
    base.check_decode(a, q, 0.2, True)


@pytest.mark.parametrize("G", [2, 9])
def test_weights_of_whole_and_of_cut_rows(G):
    """bf16, head dim 128: the attention adds the weights of rows of 1,024 slots or more that one CTA did, the second
    kernel those of shorter rows and of rows that several CTAs share.  Every row's weights are added once."""
    B, H, d, cap = 60, 8, 128, 1600
    kinds = (1023, 1024, 1025, 1500, 300, 1600, 1024, 1023)
    counts = [[kinds[(b + 3 * h) % 8] for h in range(H)] for b in range(B)]
    a = ref.make_cache(B, H, d, 64, cap, seed=G)
    base.fill_random(a, counts, seed=G)
    q = (2 * torch.randn(B, G * H, d, generator=gen(1))).to(torch.bfloat16).cuda()
    got = decode_launches(a, q, True)
    assert len(got) == 2 and "paged_decode_kernelILi128ELb0E" in got[0][0] and "paged_join_kernel" in got[1][0]
    # The rows in a line, each as its blocks of 128 slots and two more, cut into equal shares.
    sizes = [-(-n // 128) + 2 for row in counts for n in row]
    share, at, found = -(-sum(sizes) // got[0][1]), 0, set()
    for size, n in zip(sizes, (n for row in counts for n in row)):
        whole = (at + 2) // share == (at + size - 1) // share
        found.add(("whole, long" if n >= 1024 else "whole, short") if whole else "cut")
        at += size
    assert found == {"whole, long", "whole, short", "cut"}
    base.check_decode(a, q, 1 / math.sqrt(d), True)


def test_debug_build_in_bounds(word):  # noqa: F811
    test_shares_of_more_rows_than_are_held("e4m3", 12)
    test_weights_of_whole_and_of_cut_rows(2)
    test_weights_of_whole_and_of_cut_rows(9)
    torch.cuda.synchronize()
    code = int(word.item())
    assert code == 0, f"bounds check failed: kernel {(code >> 16) & 0xff}, site {(code >> 8) & 0xff}"
