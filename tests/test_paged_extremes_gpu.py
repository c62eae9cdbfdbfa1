"""The paged cache at the ends of what its entry points take: capacities of one to seven slots, pages of 1,024, the
largest group, the most heads, the largest batches."""
import math

import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base
from test_paged_limits_gpu import word  # noqa: F401

pytestmark = pytest.mark.gpu
gen = base.gen


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("cap", [1, 2, 3, 5, 7])
def test_a_few_slots(cap, dtype):
    """Compaction, appends by both calls and attention in rows of less than a page."""
    a = ref.make_cache(2, 2, 64, 8, cap, dtype, seed=cap)
    k, v = (torch.randn(9, 2, 64, generator=gen(s)).to(torch.bfloat16) for s in (1, 2))
    want = ref.compact(a, k, v, None, [0, cap + 1, 9], None)
    kv.paged_compact_kv(k.cuda(), v.cuda(), None, [0, cap + 1, 9], kv.PagedCache(**a))
    ref.assert_same_state(a, want)
    for step in range(4):
        base.check_append(a, None if step % 2 else [0, 1, 1 + step // 2], 0, 0, seed=step)
        q = torch.randn(2, 6, 64, generator=gen(step)).to(torch.bfloat16).cuda()
        base.check_decode(a, q, 0.3, True)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("e4m3", 64)])
def test_pages_of_1024_slots(dtype, d):
    a = ref.make_cache(2, 2, d, 1024, 3000, dtype, "phd", seed=1)
    k, v = (torch.randn(5000, 2, d, generator=gen(s)).to(torch.bfloat16) for s in (1, 2))
    score = torch.rand(2, 5000, generator=gen(3))
    want = ref.compact(a, k, v, None, [0, 3100, 5000], score)
    kv.paged_compact_kv(k.cuda(), v.cuda(), None, [0, 3100, 5000], kv.PagedCache(**a), score=score.cuda())
    ref.assert_same_state(a, want)
    base.check_append(a, None, 64, 4, seed=1)
    base.check_append(a, [0, 20, 60], 64, 4, seed=2)
    base.check_decode(a, torch.randn(2, 6, d, generator=gen(4)).to(torch.bfloat16).cuda(), 0.1, True)


@pytest.mark.parametrize("cap,dtype,accumulate", [(70, "bf16", False), (70, "e4m3", True), (1100, "bf16", True)])
def test_the_largest_group(cap, dtype, accumulate):
    """1,024 query heads per KV head: 64 chunks of 16."""
    a = ref.make_cache(1, 2, 64, 16, cap, dtype, seed=cap)
    base.fill_random(a, [[cap, cap // 3]], seed=cap)
    q = torch.randn(1, 2048, 64, generator=gen(1)).to(torch.bfloat16).cuda()
    base.check_decode(a, q, 0.2, accumulate)


def test_the_most_kv_heads():
    a = ref.make_cache(1, 1024, 64, 8, 20, seed=1)
    base.fill_random(a, [[(h * 5) % 21 for h in range(1024)]], seed=1)
    base.check_append(a, None, 4, 2, seed=1)
    base.check_append(a, [0, 3], 4, 2, seed=2)
    base.check_decode(a, torch.randn(1, 1024, 64, generator=gen(1)).to(torch.bfloat16).cuda(), 0.2, True)


def test_the_largest_packed_batch():
    """512 sequences, some without a token: compaction and several tokens each."""
    lens = [(5 * b) % 23 for b in range(512)]
    cu = base.np.concatenate([[0], base.np.cumsum(lens)]).tolist()
    a = ref.make_cache(512, 1, 64, 8, 16, seed=1)
    k, v = (torch.randn(cu[-1], 1, 64, generator=gen(s)).to(torch.bfloat16) for s in (1, 2))
    want = ref.compact(a, k, v, None, cu, None)
    kv.paged_compact_kv(k.cuda(), v.cuda(), None, cu, kv.PagedCache(**a))
    ref.assert_same_state(a, want)
    base.check_append(a, base.np.concatenate([[0], base.np.cumsum([b % 5 for b in range(512)])]).tolist(), 4, 2, seed=1)


def test_the_largest_batch():
    """65,535 sequences: one token each, over the least weight; attention over rows on shared pages, most of them empty."""
    B, d = 65535, 64
    g = gen(1)
    a = ref.make_cache(B, 1, d, 8, 8, seed=1)
    table = a["page_table"][:, 0].long()
    for name in ("k_pages", "v_pages"):
        a[name].copy_(torch.randn(a[name].shape, generator=g))
    a["weight"].copy_(torch.rand(a["weight"].shape, generator=g))
    a["pos"].copy_(torch.arange(8, dtype=torch.int32).expand(a["pos"].shape))
    a["count"].fill_(8)
    a["seen"].fill_(8)
    x = torch.randn(B, 2, d, generator=g).to(torch.bfloat16).cuda()
    k, v, pos, weight = (a[n][table, 0].clone() for n in ("k_pages", "v_pages", "pos", "weight"))
    slot = weight.argmin(1)
    got = kv.paged_append_kv(x[:, :1], x[:, 1:], kv.PagedCache(**a), 0, 0)
    at = torch.arange(B, device="cuda")
    assert torch.equal(got[:, 0], slot.int())                    # the position of slot c is c
    k[at, slot], v[at, slot], pos[at, slot], weight[at, slot] = x[:, 0], x[:, 1], 8, 0.0
    for name, want in (("k_pages", k), ("v_pages", v), ("pos", pos), ("weight", weight)):
        assert torch.equal(a[name][table, 0], want), name
    assert a["count"].eq(8).all() and a["seen"].eq(9).all()

    cap = 1100
    shared = ref.make_cache(11, 1, d, 64, cap, seed=2, weight=False)
    base.fill_random(shared, [[cap]] * 11, seed=2)
    big = dict(shared, page_table=shared["page_table"][torch.arange(B) % 11].contiguous(),
               count=torch.where(torch.rand(B, 1, generator=g) < 0.01, torch.randint(1, cap + 1, (B, 1), generator=g),
                                 0).to(torch.int32).cuda(), seen=None, pos=None)
    big["count"][0], big["count"][-1] = cap, cap - 1
    q = torch.randn(B, 2, d, generator=g).to(torch.bfloat16).cuda()
    out, lse = kv.paged_decode_attention(q, kv.PagedCache(**big), scale=1 / math.sqrt(d))
    empty = big["count"][:, 0] == 0
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()
    some = torch.cat([torch.tensor([0, B - 1], device="cuda"), (~empty).nonzero()[1:120, 0]])
    few = dict(big, page_table=big["page_table"][some].contiguous(), count=big["count"][some].contiguous())
    want, want_lse, tol, tol_lse, _ = ref.decode(q[some], few, 1 / math.sqrt(d))
    assert (abs(out[some].double().cpu().numpy() - want) <= tol).all()
    assert (abs(lse[some].double().cpu().numpy() - want_lse) <= tol_lse).all()


def test_debug_build_in_bounds(word):  # noqa: F811
    for cap in (1, 3, 7):
        test_a_few_slots(cap, "e4m3")
    test_pages_of_1024_slots("bf16", 128)
    test_the_largest_group(1100, "bf16", True)
    test_the_most_kv_heads()
    test_the_largest_packed_batch()
    test_the_largest_batch()
    torch.cuda.synchronize()
    code = int(word.item())
    assert code == 0, f"bounds check failed: kernel {(code >> 16) & 0xff}, site {(code >> 8) & 0xff}"
