"""The paged cache at its edges: pools past 4 GiB, K and V in one pool, shared pages, many sequences, calls at once
on two streams, a process's first call captured in a graph, and the debug build's bounds checks."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref
import test_paged_cache_gpu as base
from future_attention_targets_b200 import _binding as B
from future_attention_targets_b200.build import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
gen = base.gen


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_pools_past_4_gib(dtype):
    """Pages whose byte offsets need more than 32 bits: compaction, append and attention."""
    H, d, page, cap = 8, 128, 64, 1000
    dt = ref.E4M3 if dtype == "e4m3" else torch.bfloat16
    N = (5 << 30) // (H * page * d * (1 if dtype == "e4m3" else 2))
    a = ref.make_cache(1, H, d, page, cap, dtype, seed=1)
    a["k_pages"], a["v_pages"] = (torch.empty(N, H, page, d, dtype=dt, device="cuda") for _ in range(2))
    a["pos"] = torch.full((N, H, page), -7, dtype=torch.int32, device="cuda")
    a["weight"] = torch.zeros(N, H, page, device="cuda")
    a["page_table"] = (N - 1 - 3 * torch.arange(16, dtype=torch.int32)).view(1, 16).cuda()
    T = 990
    k, v = (torch.randn(T, H, d, generator=gen(s)).to(torch.bfloat16) for s in (1, 2))
    score = torch.rand(H, T, generator=gen(3))
    kv.paged_compact_kv(k.cuda(), v.cuda(), None, [0, T], kv.PagedCache(**a), score=score.cuda())
    k_rows, v_rows = ref.get_rows(a, 0, 5, T)
    scale = [float(a[n][5]) if a.get(n) is not None else 1.0 for n in ("k_scale", "v_scale")]
    for got, src, sc in ((k_rows, k, scale[0]), (v_rows, v, scale[1])):
        want = ref.quantise(src[:, 5], dt, sc).float().double().numpy() * (sc if dtype == "e4m3" else 1.0)
        assert np.array_equal(got, want)
    x = torch.randn(20, 2 * H, d, generator=gen(4)).to(torch.bfloat16).cuda()
    cache = kv.PagedCache(**a)
    kv.paged_append_kv(x[:, :H], x[:, H:], cache, 64, 4, cu_new=[0, 20])
    kv.paged_append_kv(x[:1, :H], x[:1, H:], cache, 64, 4)
    assert a["count"].tolist() == [[1000] * H] and a["seen"].tolist() == [[1011] * H]
    q = torch.randn(1, 4 * H, d, generator=gen(5)).to(torch.bfloat16).cuda()
    base.check_decode(a, q, 1 / math.sqrt(d), True)


def test_k_and_v_side_by_side_in_one_pool():
    """[n_pages, 2, H, page, d] and [n_pages, page, 2, H, d]: the same results as separate pools."""
    d, H, page, cap = 64, 3, 16, 200
    a = ref.make_cache(2, H, d, page, cap, seed=4)
    base.fill_random(a, [[200, 100, 7], [0, 199, 200]], seed=4)
    q = torch.randn(2, 12, d, generator=gen(1)).to(torch.bfloat16).cuda()
    out, lse = kv.paged_decode_attention(q, kv.PagedCache(**a))
    k, v = a["k_pages"], a["v_pages"]
    for pool, views in ((torch.stack([k, v], 1), lambda p: (p[:, 0], p[:, 1])),
                        (torch.stack([k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)], 2),
                         lambda p: (p[:, :, 0].permute(0, 2, 1, 3), p[:, :, 1].permute(0, 2, 1, 3)))):
        c = dict(a)
        c["k_pages"], c["v_pages"] = views(pool)
        c["pos"], c["weight"], c["count"], c["seen"] = (a[n].clone() for n in ("pos", "weight", "count", "seen"))
        o2, l2 = kv.paged_decode_attention(q, kv.PagedCache(**c))
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        base.check_append(c, None, 8, 4, seed=1)
        base.check_append(c, [0, 5, 8], 8, 4, seed=2)


def test_sequences_share_the_pages_of_a_prefix():
    a = ref.make_cache(3, 2, 64, 16, 100, seed=4, weight=False)
    base.fill_random(a, [[90, 90]] * 3, seed=4)
    a["page_table"][1:, :5] = a["page_table"][0, :5]
    q = torch.randn(3, 4, 64, generator=gen(1)).to(torch.bfloat16).cuda()
    base.check_decode(a, q, 0.2, False)


def test_more_sequences_than_a_packed_call_takes():
    """600 sequences: one token each, and attention; with cu_new the call is refused."""
    B_, H, cap = 600, 2, 40
    counts = [[(b * 7 + h) % 41 for h in range(H)] for b in range(B_)]
    a = ref.make_cache(B_, H, 64, 8, cap, seed=1)
    base.fill_random(a, counts, seed=2)
    base.check_append(a, None, 4, 2, seed=1)
    q = torch.randn(B_, 2 * H, 64, generator=gen(1)).to(torch.bfloat16).cuda()
    base.check_decode(a, q, 0.2, True)
    x = torch.zeros(1, H, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kv.KvpopError, match="512"):
        kv.paged_append_kv(x, x, kv.PagedCache(**a), 4, 2, cu_new=[0] * B_ + [1])


@pytest.mark.parametrize("dtype,G", [("bf16", 2), ("e4m3", 12)])
def test_attention_over_more_rows_than_are_held(dtype, G):
    """More than 1,024 rows that are dealt out in shares, most of them short or empty."""
    B_, H, cap = 270, 4, 700
    rng = np.random.default_rng(3)
    counts = np.where(rng.random((B_, H)) < 0.05, 700, rng.integers(-1, 5, (B_, H))).tolist()
    a = ref.make_cache(B_, H, 64, 64, cap, dtype, seed=1)
    base.fill_random(a, counts, seed=2)
    q = torch.randn(B_, G * H, 64, generator=gen(1)).to(torch.bfloat16).cuda()
    base.check_decode(a, q, 0.2, True)


def test_all_rows_empty():
    for cap in (100, 2000):
        a = ref.make_cache(3, 2, 64, 16, cap, seed=1)
        a["count"].copy_(torch.tensor([[0, -1], [0, 0], [-5, 0]]))
        q = torch.randn(3, 8, 64, generator=gen(1)).to(torch.bfloat16).cuda()
        out, lse = base.check_decode(a, q, 0.2, True)
        assert not out.any() and torch.isneginf(lse).all()


def test_no_tokens():
    a = ref.make_cache(2, 1, 64, 8, 16, seed=1)
    a["count"].fill_(9)
    empty = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv.paged_compact_kv(empty, empty, None, [0, 0, 0], kv.PagedCache(**a))
    assert a["count"].tolist() == [[0], [0]] and a["seen"].tolist() == [[0], [0]]
    assert kv.paged_append_kv(empty, empty, kv.PagedCache(**a), 4, 2, cu_new=[0, 0, 0]).shape == (0, 1)


def test_one_token_by_either_call():
    """A chunk of one token per sequence does what the call without cu_new does."""
    states = []
    for cu in (None, [0, 1, 2, 3]):
        a = ref.make_cache(3, 2, 128, 16, 3000, seed=1)
        base.fill_random(a, [[3000, 3000], [2999, 3000], [0, -1]], seed=2)
        for step in range(3):
            base.check_append(a, cu, 64, 4, seed=step)
        states.append({n: a[n].cpu() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")})
    ref.assert_same_state(states[0], states[1])


def test_two_threads_on_two_streams():
    """Calls at once, each with its own cache, buffers and stream, give what they give one by one."""
    def make(seed):
        a = ref.make_cache(2, 2, 128, 16, 1500, seed=seed)
        base.fill_random(a, [[1500, 700], [1500, 1500]], seed=seed)
        x = torch.randn(2, 12, 128, generator=gen(seed)).to(torch.bfloat16).cuda()
        return a, x

    def steps(a, x, stream):
        cache, outs = kv.PagedCache(**a), []
        for _ in range(20):
            kv.paged_append_kv(x[:, 8:10], x[:, 10:], cache, 64, 4, stream=stream)
            outs.append(kv.paged_decode_attention(x[:, :8], cache, accumulate=True, stream=stream))
        return outs

    alone = []
    for seed in (1, 2):
        a, x = make(seed)
        alone.append((steps(a, x, None), a))
    torch.cuda.synchronize()
    pairs, got = [make(1), make(2)], [None, None]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        got[i] = steps(*pairs[i], s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        for (o, l), (o2, l2) in zip(alone[i][0], got[i]):
            assert torch.equal(o, o2) and torch.equal(l, l2)
        ref.assert_same_state(pairs[i][0], {n: alone[i][1][n].cpu() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")})


def test_eight_bits_without_scales():
    """No scales are scales of 1, each on its own."""
    for drop in (("k_scale", "v_scale"), ("k_scale",), ("v_scale",)):
        a = ref.make_cache(2, 2, 64, 16, 600, "e4m3", seed=3)
        for name in drop:
            a[name] = None
        T = 700
        k, v = (torch.randn(T, 2, 64, generator=gen(s)).to(torch.bfloat16) for s in (1, 2))
        want = ref.compact(a, k, v, None, [0, 500, T], None)
        kv.paged_compact_kv(k.cuda(), v.cuda(), None, [0, 500, T], kv.PagedCache(**a))
        ref.assert_same_state(a, want)
        base.check_append(a, None, 16, 4, seed=1)
        base.check_append(a, [0, 3, 9], 16, 4, seed=2)
        q = torch.randn(2, 6, 64, generator=gen(5)).to(torch.bfloat16).cuda()
        base.check_decode(a, q, 0.3, True)


def test_binding_refuses():
    """Wrong types, shapes, layouts and sizes raise before anything is enqueued, and change nothing."""
    a = ref.make_cache(2, 2, 64, 16, 100, seed=1)
    base.fill_random(a, [[100, 20], [0, 5]], seed=1)
    before = {n: ref.as_bytes(a[n]).copy() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")}
    cache = kv.PagedCache(**a)
    dev = "cuda"
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    kn = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=dev)
    T = 30
    k = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device=dev)
    keep, score = torch.ones(2, T, dtype=torch.uint8, device=dev), torch.zeros(2, T, device=dev)
    wide = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=dev)
    bad_caches = [
        dict(k_pages=a["k_pages"].float()), dict(v_pages=a["v_pages"][:-1]), dict(k_pages=a["k_pages"][..., ::2]),
        dict(k_pages=a["k_pages"][:1].expand(a["k_pages"].shape)), dict(page_table=a["page_table"].long()),
        dict(page_table=a["page_table"][:, ::2]), dict(count=a["count"][:1]), dict(count=a["count"].float()),
        dict(seen=a["seen"].cpu()), dict(pos=a["pos"].long()), dict(weight=a["weight"].double()), dict(capacity=0),
        dict(capacity=10 ** 6), dict(k_scale=torch.ones(2, device=dev)),
    ]
    for kw in bad_caches:
        with pytest.raises((TypeError, ValueError)):
            kv.PagedCache(**{**a, **kw})
    decode, append, compact = kv.paged_decode_attention, kv.paged_append_kv, kv.paged_compact_kv
    no_weight = kv.PagedCache(**{**a, "weight": None})
    small = torch.empty(16, dtype=torch.uint8, device=dev)
    bad_calls = [
        lambda: decode(q.float(), cache), lambda: decode(q[:1], cache), lambda: decode(q[:, :3], cache),
        lambda: decode(q.cpu(), cache), lambda: decode(wide[..., ::2], cache), lambda: decode(q[:, :, :32], cache),
        lambda: decode(q, cache, out=q.float()), lambda: decode(q, cache, lse=torch.empty(2, 3, device=dev)),
        lambda: decode(q, cache, accumulate=True, workspace=small), lambda: decode(q, cache, scale=0.0),
        lambda: decode(q, cache, scale=float("inf")), lambda: decode(q, no_weight, accumulate=True),
        lambda: decode(q, cache, status=torch.zeros(1, device=dev)),
        lambda: append(kn[:1], kn, cache, 4, 2), lambda: append(kn, kn.float(), cache, 4, 2),
        lambda: append(kn, wide[:, :2, :64], cache, 4, 2), lambda: append(kn, kn, cache, -1, 2),
        lambda: append(kn, kn, cache, 100, 2), lambda: append(kn, kn, cache, 4, 2, cu_new=[0, 1]),
        lambda: append(kn, kn, cache, 4, 2, cu_new=[0, 2, 1]), lambda: append(kn, kn, cache, 1, 2, cu_new=[0, 0, 2]),
        lambda: append(kn, kn, cache, 4, 2, cu_new=[0, 2 ** 40, 2]), lambda: append(kn, kn, no_weight, 4, 2),
        lambda: append(kn, kn, cache, 4, 2, evicted=torch.empty(2, 3, dtype=torch.int32, device=dev)),
        lambda: compact(k, k[:-1], keep, [0, 10, T], cache), lambda: compact(k, k, keep[:1], [0, 10, T], cache),
        lambda: compact(k, k, keep, [0, T], cache), lambda: compact(k, k, keep, [0, 10, T - 1], cache),
        lambda: compact(k, k, keep, [0, 20, 10], cache), lambda: compact(k, k, keep.float(), [0, 10, T], cache),
        lambda: compact(k, k, keep, [0, 10, T], cache, score=score.double()),
        lambda: compact(k, k, keep, [0, 10, T], no_weight, score=score),
    ]
    for i, call in enumerate(bad_calls):
        with pytest.raises((TypeError, ValueError, kv.KvpopError)):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    for n, x in before.items():
        assert np.array_equal(ref.as_bytes(a[n]), x)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import paged_reference as ref, test_paged_cache_gpu as base
import future_attention_targets_b200 as kv
def make():
    a = ref.make_cache(2, 2, 128, 16, 1500, seed=1)
    base.fill_random(a, [[1500, 700], [1400, 1500]], seed=1)
    return a
x = torch.randn(2, 12, 128, generator=base.gen(1)).to(torch.bfloat16).cuda()
a = make()
c = kv.PagedCache(**a)
ws = torch.empty(kv.paged_decode_workspace_bytes(c, 8), dtype=torch.uint8, device="cuda")
out, lse = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")
ev = torch.empty(2, 2, dtype=torch.int32, device="cuda")
k, v = x[:, 8:10].contiguous(), x[:, 10:].contiguous()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    kv.paged_append_kv(k, v, c, 64, 4, evicted=ev)
    kv.paged_append_kv(k, v, c, 64, 4, cu_new=[0, 1, 2], evicted=ev)
    kv.paged_decode_attention(x[:, :8], c, accumulate=True, out=out, lse=lse, workspace=ws)
g.replay()
torch.cuda.synchronize()
b = make()
d = kv.PagedCache(**b)
kv.paged_append_kv(k, v, d, 64, 4)
e2 = kv.paged_append_kv(k, v, d, 64, 4, cu_new=[0, 1, 2])
o2, l2 = kv.paged_decode_attention(x[:, :8], d, accumulate=True)
torch.cuda.synchronize()
assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(ev, e2)
ref.assert_same_state(a, {{n: b[n].cpu() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")}})
print("captured first")
"""


def test_first_call_of_a_process_is_captured():
    code = FIRST_CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured first" in got.stdout, got.stdout + got.stderr


@pytest.fixture
def word():
    """The debug build, with a registered, zero-filled word, for one test."""
    old = B.use_library(build(debug=True))
    w = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.debug_set_word(w)
    try:
        yield w
    finally:
        B.debug_set_word(None)
        B.use_library(old)


def test_debug_build_finds_every_index_in_bounds(word):
    for case in base.CASES:
        base.test_decode_small(case, True)
    base.test_decode_many_splits(20, 8, 16, 128, 16, 1100, "bf16", 6)
    base.test_decode_many_splits(3, 8, 5, 128, 128, 9001, "e4m3", 4)
    base.test_compact((3001, 17, 1024, 1025), 2, 128, 64, 900, "bf16", "phd", 0.35, "score")
    base.test_compact((5, 2047, 2048, 2049), 1, 64, 128, 3000, "e4m3", "phd", 1.0, "mask")
    base.test_append_one(2, 2, 64, 16, 100, [[100, 99], [0, 50]], 8, 4, "bf16", "hpd")
    base.test_append_one(60, 8, 64, 8, 40, [[40] * 8] * 60, 4, 2, "e4m3", "phd")
    base.test_append_chunk(2, 2, 64, 32, 20000, [[20000, 19990], [5000, 20000]], [700, 650], 1000, 16, "bf16")
    base.test_append_chunk(1, 3, 64, 8, 48, [[48, 47, -1]], [44], 44, 4, "e4m3")
    base.test_prompt_to_decoding("bf16")
    torch.cuda.synchronize()
    code = int(word.item())
    assert code == 0, f"bounds check failed: kernel {(code >> 16) & 0xff}, site {(code >> 8) & 0xff}"
