"""e4m3 caches with scales far from 1: a power of two in a scale is a power of two in the result, bit for bit."""
import math

import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base

pytestmark = pytest.mark.gpu
gen = base.gen


def results(power_k, power_v, cap, d, G):
    a = ref.make_cache(2, 2, d, 16, cap, "e4m3", seed=3)
    a["k_scale"].mul_(2.0 ** power_k)
    a["v_scale"].mul_(2.0 ** power_v)
    base.fill_random(a, [[cap, cap // 2], [cap - 1, 17]], seed=9)
    q = torch.randn(2, 2 * G, d, generator=gen(2)).to(torch.bfloat16).mul(2.0 ** -power_k).cuda()
    out, lse = kv.paged_decode_attention(q, kv.PagedCache(**a), scale=1 / math.sqrt(d), accumulate=True)
    return out.float().cpu().double(), lse.cpu(), a["weight"].cpu()


@pytest.mark.parametrize("cap,d,G", [(300, 128, 4), (600, 128, 4), (600, 64, 12), (2000, 64, 3)])
@pytest.mark.parametrize("power_k,power_v", [(0, -118), (0, -60), (0, 60), (0, 118), (-100, 0), (100, 0)])
def test_powers_of_two_in_the_scales(power_k, power_v, cap, d, G):
    out, lse, weight = results(0, 0, cap, d, G)
    out2, lse2, weight2 = results(power_k, power_v, cap, d, G)
    want = out * 2.0 ** power_v
    sure = want.abs() >= 2.0 ** -126                       # smaller ones are rounded once more
    assert sure.double().mean() > 0.9
    assert torch.equal(out2[sure], want[sure])
    assert torch.equal(lse, lse2) and ref.np.array_equal(ref.as_bytes(weight), ref.as_bytes(weight2))
