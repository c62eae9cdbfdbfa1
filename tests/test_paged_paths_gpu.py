"""Appending where the sizes of the other tests pass by: each kernel and each way of dealing rows out that the launch
chooses by size, and counts far past the capacity."""
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


def append_launch(a, cu, window, sinks):
    """(name, CTAs, threads) of the kernel that such an append launches."""
    B, H = a["count"].shape
    T = B if cu is None else cu[-1]
    x = torch.zeros(T, H, a["k_pages"].shape[3], dtype=torch.bfloat16, device="cuda")
    cache, evicted = kv.PagedCache(**a), torch.empty(T, H, dtype=torch.int32, device="cuda")
    got = launches(lambda s: kv.paged_append_kv(x, x, cache, window, sinks, cu_new=cu, evicted=evicted, stream=s))
    assert len(got) == 1
    return got[0]


def name_of(d, dtype, rest):
    return f"paged_append_kernelILi{d}ELb{int(dtype == 'e4m3')}E{rest}"


def running(m):
    return [0, *np.cumsum(m).tolist()]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_one_token_streamed_with_head_dim_128(dtype):
    """More than 444 rows of 128 dims: every lane of warp 0 carries a word of the new rows."""
    B, H, cap = 115, 4, 40
    counts = [[(cap, cap - 1, cap, 0, 17, -1, cap)[(b * H + h) % 7] for h in range(H)] for b in range(B)]
    a = ref.make_cache(B, H, 128, 8, cap, dtype, "phd", seed=cap)
    base.fill_random(a, counts, seed=1)
    name, ctas, _ = append_launch(a, None, 8, 2)
    assert f"paged_append_stream_kernelILi128ELb{int(dtype == 'e4m3')}E" in name and ctas < B * H
    for step in range(3):
        base.check_append(a, None, 8, 2, seed=step, fused=step == 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_several_tokens_into_many_short_rows(dtype, d):
    """The 256-thread kernel: more CTAs than two per SM, short slices."""
    B, H, cap = 75, 5, 100
    counts = [[(cap, cap, cap - 3, 5, -1, cap)[(b * H + h) % 6] for h in range(H)] for b in range(B)]
    a = ref.make_cache(B, H, d, 16, cap, dtype, seed=d)
    base.fill_random(a, counts, seed=d)
    cu = running([(3 * b) % 9 for b in range(B)])
    name, ctas, threads = append_launch(a, cu, 8, 4)
    assert name_of(d, dtype, "Lb1ELi256E") in name and (ctas, threads) == (B * H, 256)
    for step in range(2):
        base.check_append(a, cu, 8, 4, seed=step, fused=step == 1)


@pytest.mark.parametrize("B", [9, 320])
def test_sequences_with_one_token_or_none(B):
    """A step in which some sequences are idle, few rows and many."""
    a = ref.make_cache(B, 2, 64, 8, 60, seed=B)
    base.fill_random(a, [[(60, 59, 60, 3, -1)[(2 * b + h) % 5] for h in range(2)] for b in range(B)], seed=B)
    for step in range(3):
        base.check_append(a, running([int((b + step) % 3 > 0) for b in range(B)]), 8, 2, seed=step)


def test_several_tokens_into_many_long_rows():
    """Rows over 16,384 slots, more than 74 of them: two CTAs per row, slices over 8,192 slots."""
    B, cap = 76, 16400
    a = ref.make_cache(B, 1, 64, 64, cap, seed=1)
    base.fill_random(a, [[cap - (b % 5)] for b in range(B)], seed=1)
    cu = running([(7 * b) % 33 for b in range(B)])
    name, ctas, threads = append_launch(a, cu, 32, 4)
    assert name_of(64, "bf16", "Lb1ELi512E") in name and (ctas, threads) == (2 * B, 512)
    base.check_append(a, cu, 32, 4, seed=1)


def test_one_token_into_slices_of_several_rounds():
    """Slices over 4,096 slots: a thread's second round asks for its page numbers itself.  The least weights lie there."""
    cap, slice_ = 40100, 5016
    a = ref.make_cache(1, 2, 64, 64, cap, seed=1)
    base.fill_random(a, [[cap, cap]], seed=1)
    name, ctas, threads = append_launch(a, None, 64, 4)
    assert name_of(64, "bf16", "Lb0ELi256E") in name and (ctas, threads) == (16, 256)
    pg, off = (x.cuda() for x in ref.slots_of(a, 0, cap, 64))
    least = [c * slice_ + 4096 + at for c, at in ((3, 0), (0, 1), (6, 919), (7, 890), (2, 5), (5, 411))]
    for h in range(2):
        for i, c in enumerate(least):
            a["weight"][pg[c], h, off[c]] = -6.0 + (i if h == 0 else -i)
            a["pos"][pg[c], h, off[c]] = 200000 + c                     # none of them a sink
    a["seen"].fill_(300000)
    for step in range(len(least)):
        base.check_append(a, None, 64, 4, seed=step)
    for h in range(2):
        assert a["pos"][pg[least], h, off[least]].ge(300000).all()      # they have all gone


@pytest.mark.parametrize("weights", ["distinct", "equal"])
def test_more_victims_in_a_slice_than_its_list_holds(weights):
    """2,490 victims in the first slice of 2,504 slots: the row list, of 2,048 entries, is filled twice."""
    cap, m = 20000, 2490
    a = ref.make_cache(1, 1, 64, 64, cap, seed=1)
    base.fill_random(a, [[cap]], seed=1)
    assert append_launch(a, [0, m], m, 4)[1] == 8
    pg, off = (x.cuda() for x in ref.slots_of(a, 0, 2504, 64))
    a["weight"][pg, 0, off] = torch.rand(2504, generator=gen(3)).cuda() - 2 if weights == "distinct" else -1.0
    base.check_append(a, [0, m], m, 4, seed=1)


def test_more_free_slots_in_a_share_than_its_list_holds():
    """17,000 tokens into an empty row of eight CTAs: shares of 2,125 rows, over two fillings of the list."""
    cap, m = 20000, 17000
    a = ref.make_cache(1, 1, 64, 64, cap, seed=1)
    assert append_launch(a, [0, m], m, 4)[1] == 8
    base.check_append(a, [0, m], m, 4, seed=1)
    base.check_append(a, [0, 4000], m, 4, seed=2)         # the rest of the free slots and 1,000 victims


@pytest.mark.parametrize("B,cu", [(450, None), (2, None), (3, [0, 2, 2, 5])], ids=["many rows", "few rows", "several tokens"])
def test_counts_past_the_capacity_mean_full_rows(B, cu):
    """A count beyond the capacity, the largest int32 too, is a full row, and its count is the capacity afterwards."""
    a = ref.make_cache(B, 1, 64, 8, 40, seed=1)
    base.fill_random(a, [[40 + (b % 3)] for b in range(B)], seed=2)
    a["count"][::2] = 2 ** 31 - 1
    base.check_append(a, cu, 8, 2, seed=3)
    touched = [b for b in range(B) if cu is None or cu[b + 1] > cu[b]]
    assert a["count"].cpu()[touched].eq(40).all()


def test_debug_build_in_bounds(word):  # noqa: F811
    test_one_token_streamed_with_head_dim_128("e4m3")
    test_several_tokens_into_many_short_rows("bf16", 128)
    test_several_tokens_into_many_short_rows("e4m3", 64)
    test_sequences_with_one_token_or_none(320)
    test_several_tokens_into_many_long_rows()
    test_one_token_into_slices_of_several_rounds()
    test_more_victims_in_a_slice_than_its_list_holds("equal")
    test_more_free_slots_in_a_share_than_its_list_holds()
    torch.cuda.synchronize()
    code = int(word.item())
    assert code == 0, f"bounds check failed: kernel {(code >> 16) & 0xff}, site {(code >> 8) & 0xff}"
