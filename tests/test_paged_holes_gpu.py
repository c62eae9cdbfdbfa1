"""Appending to rows whose page table has an entry outside the pool: no slot of that page goes, nothing is written
there, the status word says so, and everything else is as if those slots could not go."""
import numpy as np
import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,m", [(150, None), (4, None), (4, 3), (111, 3)],
                         ids=["streamed", "a cluster per row", "several tokens", "several tokens, many rows"])
def test_append_around_a_hole(B, m, dtype):
    H, cap, page, window, sinks = 3, 300, 16, 16, 4
    a = ref.make_cache(B, H, 64, page, cap, dtype, seed=B, spare=4)
    base.fill_random(a, [[cap] * H if b % 7 != 3 else [cap - 1, 40, -1] for b in range(B)], seed=B)
    holes = {(1, 2): -1, (B - 2, 18): a["k_pages"].shape[0], (2, 0): 2 ** 31 - 1}
    # The slots behind the holes weigh least: they would go first.
    spare = sorted(set(range(a["k_pages"].shape[0])) - set(a["page_table"].flatten().tolist()))
    for (b, e) in holes:
        a["weight"][a["page_table"][b, e].long()] = -1e9
    # The reference's table names a spare page there, whose positions say that none of its slots may go.
    want_from = dict(a, page_table=a["page_table"].clone())
    for (b, e), page_of_none in zip(holes, spare):
        want_from["page_table"][b, e] = page_of_none
        a["pos"][page_of_none] = -1
    for (b, e), entry in holes.items():
        a["page_table"][b, e] = entry
    cu = None if m is None else [m * b for b in range(B + 1)]
    T = B if m is None else m * B
    x = (3 * torch.randn(T, 2 * H, 64, generator=base.gen(1))).to(torch.bfloat16)
    for step in range(2):
        want, evicted = ref.append(want_from, x[:, :H], x[:, H:], list(range(B + 1)) if cu is None else cu, window, sinks)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = kv.paged_append_kv(x[:, :H].cuda().contiguous(), x[:, H:].cuda().contiguous(), kv.PagedCache(**a), window, sinks,
                                 cu_new=cu, status=status)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), evicted)
        ref.assert_same_state(a, want)
        with pytest.raises(kv.KvpopError) as error:
            kv.check_status(status)
        assert error.value.status == 5                    # KVPOP_ERR_BOUNDS
