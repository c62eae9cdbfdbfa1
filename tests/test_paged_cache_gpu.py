"""The paged key-value cache on the GPU against the 64-bit reference: compaction and append bit for bit, decode
attention within bounds derived in paged_reference.decode."""
import math

import numpy as np
import pytest
import torch

import future_attention_targets_b200 as kv
import paged_reference as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def fill_random(a, counts, seed, gain=1.0, shuffle=True):
    """Random rows, distinct positions and heavy-tailed weights in the slots in use of every row."""
    g = gen(seed)
    B, H = a["count"].shape
    d, cap = a["k_pages"].shape[3], a["capacity"]
    for b in range(B):
        for h in range(H):
            n = counts[b][h]
            a["count"][b, h] = n
            n = min(max(n, 0), cap)
            a["seen"][b, h] = 3 * n + 2
            if n == 0:
                continue
            eight = a["k_pages"].dtype == ref.E4M3
            k = torch.randn(n, d, generator=g) * gain * (50 if eight else 1)
            v = torch.randn(n, d, generator=g) * (60 if eight else 1)
            pos = torch.sort(torch.randperm(3 * n + 2, generator=g)[:n]).values
            if shuffle:
                pos = pos[torch.randperm(n, generator=g)]
            ref.set_rows(a, b, h, k, v, pos, torch.exp(2 * torch.randn(n, generator=g)) if a.get("weight") is not None else None)


def check_decode(a, q, scale, accumulate, bad=(), **kw):
    out, lse, tol_out, tol_lse, add = ref.decode(q, a, scale, bad)
    before = None if a.get("weight") is None else a["weight"].clone()
    cache = kv.PagedCache(**a)
    got, got_lse = kv.paged_decode_attention(q, cache, scale=scale, accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    g, gl = got.float().cpu().double().numpy(), got_lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(lse))
    fine = np.isfinite(lse)
    over = np.abs(g - out) / np.maximum(tol_out, 1e-30)
    assert np.all(np.abs(g - out) <= tol_out), f"out off by {np.nanmax(over):.2f} of its bound"
    assert np.all(np.abs(gl[fine] - lse[fine]) <= tol_lse[fine])
    if before is None:
        return got, got_lse
    page = a["k_pages"].shape[2]
    want, tol = before.cpu().double().clone(), torch.zeros(before.shape, dtype=torch.float64)
    if accumulate:
        for (b, h), (w, t) in add.items():
            use = [c for c in range(len(w)) if (b, c // page) not in bad]
            pg, off = (x[use] for x in ref.slots_of(a, b, len(w), page))
            want[pg, h, off] += torch.from_numpy(w)[use]
            tol[pg, h, off] = torch.from_numpy(t)[use] + 2 * ref.EPS32 * want[pg, h, off].abs()
    now = a["weight"].cpu().double()
    ok = ((now - want).abs() <= tol) | (now.isnan() & want.isnan())
    assert bool(ok.all()), f"{int((~ok).sum())} weights out of bounds"
    return got, got_lse


CASES = [
    # B, Hkv, G, d, page, cap, counts (per row or one list for all), dtype, layout
    (1, 1, 1, 64, 8, 8, [[1]], "bf16", "hpd"),
    (2, 2, 2, 64, 16, 200, [[200, 1], [0, 77]], "bf16", "hpd"),
    (3, 2, 4, 128, 64, 300, [[15, 16], [17, 300], [-1, 0]], "bf16", "hpd"),
    (2, 3, 5, 128, 8, 130, [[7, 8, 9], [129, 130, 31]], "bf16", "phd"),
    (1, 2, 3, 128, 32, 1000, [[1000, 999]], "bf16", "phd"),
    (2, 1, 7, 64, 128, 700, [[641], [500]], "bf16", "hpd"),
    (1, 2, 8, 128, 16, 517, [[517, 1]], "bf16", "hpd"),
    (2, 1, 9, 128, 16, 260, [[260], [33]], "bf16", "hpd"),
    (1, 2, 16, 64, 64, 400, [[400, 129]], "bf16", "phd"),
    (1, 1, 16, 128, 256, 513, [[513]], "bf16", "hpd"),
    (2, 1, 20, 128, 16, 150, [[150], [3]], "bf16", "hpd"),         # two head chunks, the second of four
    (1, 1, 40, 64, 32, 90, [[90]], "bf16", "hpd"),
    (2, 2, 4, 128, 64, 300, [[300, 12], [0, 299]], "e4m3", "hpd"),
    (2, 2, 7, 128, 8, 200, [[200, 199], [1, 64]], "e4m3", "phd"),
    (1, 3, 2, 64, 16, 333, [[333, 17, 16]], "e4m3", "hpd"),
    (2, 1, 12, 64, 32, 140, [[140], [131]], "e4m3", "phd"),
    (1, 1, 16, 128, 64, 300, [[300]], "e4m3", "hpd"),
    (1, 1, 4, 128, 64, 300, [[500]], "bf16", "hpd"),               # a count past the capacity
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]) + f"-{c[7]}-{c[8]}")
@pytest.mark.parametrize("accumulate", [False, True])
def test_decode_small(case, accumulate):
    B, H, G, d, page, cap, counts, dtype, layout = case
    a = ref.make_cache(B, H, d, page, cap, dtype, layout, seed=B + G + cap)
    fill_random(a, counts, seed=G * d + cap)
    q = (2 * torch.randn(B, H * G, d, generator=gen(1))).to(torch.bfloat16).cuda()
    check_decode(a, q, 1 / math.sqrt(d), accumulate)


@pytest.mark.parametrize("B,H,G,d,page,cap,dtype,seed", [
    (1, 2, 4, 128, 64, 4032, "bf16", 1), (1, 1, 2, 128, 16, 40000, "bf16", 2), (40, 4, 4, 64, 32, 3000, "bf16", 3),
    (3, 8, 5, 128, 128, 9001, "e4m3", 4), (150, 2, 1, 64, 8, 500, "e4m3", 5), (20, 8, 16, 128, 16, 1100, "bf16", 6)])
def test_decode_many_splits(B, H, G, d, page, cap, dtype, seed):
    """Several CTAs per row, ragged counts, q a slice of a fused projection."""
    rng = np.random.default_rng(seed)
    counts = np.exp(rng.uniform(0, math.log(cap), (B, H))).astype(int).tolist()
    counts[0][0] = cap
    a = ref.make_cache(B, H, d, page, cap, dtype, "hpd", seed=seed)
    fill_random(a, counts, seed)
    wide = (2 * torch.randn(B, (G + 2) * H, d, generator=gen(seed))).to(torch.bfloat16).cuda()
    check_decode(a, wide[:, :G * H], 1 / math.sqrt(d), True)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("gain,qgain", [(30.0, 20.0), (1e-3, 1e-6), (1.0, 1e4)])
def test_decode_extreme_scores(dtype, gain, qgain):
    """Softmax rows that one slot owns, and rows that are almost flat; entries of q far from 1."""
    a = ref.make_cache(1, 2, 128, 16, 600, dtype, seed=3)
    if dtype == "e4m3":
        a["k_scale"] = a["k_scale"] * gain
        fill_random(a, [[600, 311]], seed=9)
    else:
        fill_random(a, [[600, 311]], seed=9, gain=gain)
    q = (qgain * torch.randn(1, 8, 128, generator=gen(2))).to(torch.bfloat16).cuda()
    check_decode(a, q, 1 / math.sqrt(128), True)


def test_decode_infinities_and_nan_stay_in_their_rows():
    """NaN in one row's K reaches that row alone; -inf scores have probability 0; a +inf V reaches its column."""
    a = ref.make_cache(1, 4, 64, 16, 100, seed=1)
    fill_random(a, [[100, 100, 100, 100]], seed=4)
    pg, off = (x.cuda() for x in ref.slots_of(a, 0, 100, 16))
    a["k_pages"][pg[5], 1, off[5]] = float("nan")
    q = torch.randn(1, 4, 64, generator=gen(2)).abs().to(torch.bfloat16).cuda()
    a["k_pages"][pg[7], 2, off[7]] = -math.inf            # q > 0: the score is -inf
    a["v_pages"][pg[9], 3, off[9], 11] = math.inf
    out, lse = kv.paged_decode_attention(q, kv.PagedCache(**a))
    out, lse = out.float().cpu().numpy()[0], lse.cpu().numpy()[0]
    assert np.isnan(out[1]).all() and np.isnan(lse[1])
    assert np.isfinite(out[[0, 2]]).all() and np.isfinite(lse[[0, 2, 3]]).all()
    assert math.isinf(out[3, 11]) and np.isfinite(np.delete(out[3], 11)).all()


def test_decode_bad_pages_take_no_part():
    """Entries outside the pool are reported and skipped, whether or not they lie in the middle of a tile."""
    a = ref.make_cache(2, 2, 128, 8, 200, seed=6)
    fill_random(a, [[200, 150], [90, 200]], seed=6)
    a["page_table"][0, 3] = -1
    a["page_table"][1, 10] = a["k_pages"].shape[0]
    a["page_table"][1, 0] = 2 ** 31 - 1
    q = torch.randn(2, 8, 128, generator=gen(2)).to(torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_decode(a, q, 0.1, True, bad={(0, 3), (1, 10), (1, 0)}, status=status)
    with pytest.raises(kv.KvpopError) as e:
        kv.check_status(status)
    assert e.value.status == 5                            # KVPOP_ERR_BOUNDS
    # Entries behind a row's slots are not looked at.
    a["count"].fill_(20)
    a["page_table"][:, 3:] = -5
    a["page_table"][1, 0] = a["page_table"][0, 0]
    status.zero_()
    kv.paged_decode_attention(q, kv.PagedCache(**a), status=status)
    kv.check_status(status)


def test_decode_repeats_and_reuses_buffers():
    """The same bits every time, on another stream, and with a workspace full of NaN."""
    a = ref.make_cache(4, 2, 128, 16, 2000, seed=8, weight=False)
    fill_random(a, [[2000, 1500], [3, 0], [1999, 16], [700, 701]], seed=8)
    cache = kv.PagedCache(**a)
    q = torch.randn(4, 8, 128, generator=gen(2)).to(torch.bfloat16).cuda()
    out, lse = kv.paged_decode_attention(q, cache)
    need = kv.paged_decode_workspace_bytes(cache, 8)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        o2, l2 = torch.full_like(out, 5), torch.full_like(lse, 5)
        torch.cuda.synchronize()
        kv.paged_decode_attention(q, cache, out=o2, lse=l2, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


# ---------------------------------------------------------------- compaction

@pytest.mark.parametrize("lens,H,d,page,cap,dtype,layout,p", [
    ((1,), 1, 64, 8, 8, "bf16", "hpd", 1.0),
    ((300, 0, 41), 2, 64, 16, 300, "bf16", "hpd", 0.5),
    ((3001, 17, 1024, 1025), 2, 128, 64, 900, "bf16", "phd", 0.35),    # rows past the capacity
    ((700, 1300), 3, 128, 32, 2000, "e4m3", "hpd", 0.8),
    ((5, 2047, 2048, 2049), 1, 64, 128, 3000, "e4m3", "phd", 1.0),
    ((20000,), 1, 128, 16, 5000, "bf16", "hpd", 0.25),
])
@pytest.mark.parametrize("form", ["mask", "all", "score"])
def test_compact(lens, H, d, page, cap, dtype, layout, p, form):
    T, cu = sum(lens), [0, *np.cumsum(lens).tolist()]
    g = gen(T)
    k, v = (3 * torch.randn(T, H, d, generator=g).to(torch.bfloat16) for _ in range(2))
    keep = None if form == "all" else (torch.rand(H, T, generator=g) < p).to(torch.uint8) * 3
    score = torch.randn(H, T, generator=g) if form == "score" else None
    a = ref.make_cache(len(lens), H, d, page, cap, dtype, layout, seed=T)
    want = ref.compact(a, k, v, keep, cu, score)
    to = lambda t: None if t is None else t.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.paged_compact_kv(to(k), to(v), to(keep), cu, kv.PagedCache(**a), score=to(score), status=status)
    kv.check_status(status)
    ref.assert_same_state(a, want, form)


def test_compact_rounds_and_clips_to_e4m3():
    """Ties to even, values past 448, infinities and NaN, as the fp32 quotient's conversion gives them."""
    vals = torch.cat([torch.linspace(-500, 500, 1000), torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-3, 2.0 ** -10,
                      3 * 2.0 ** -11, 17.0, 19.0])]).to(torch.bfloat16)
    T = -(-len(vals) // 64)
    k = torch.zeros(T * 64, dtype=torch.bfloat16)
    k[:len(vals)] = vals
    k = k.view(T, 1, 64)
    a = ref.make_cache(1, 1, 64, 8, T, "e4m3")
    a["k_scale"].fill_(1.0)
    a["v_scale"].fill_(0.7)
    want = ref.compact(a, k, k, None, [0, T], None)
    kv.paged_compact_kv(k.cuda(), k.cuda(), None, [0, T], kv.PagedCache(**a))
    ref.assert_same_state(a, want)


@pytest.mark.parametrize("scale", [1.0, 0.7, 0.02, 3e-3, 2.0 ** -20, 1e-39, 2e38, 117.3])
def test_compact_every_bf16_value_to_e4m3(scale):
    """All 65,536 bf16 bit patterns over several scales: the rounding of the correctly rounded quotient, bit for bit."""
    k = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(1024, 1, 64)
    a = ref.make_cache(1, 1, 64, 64, 1024, "e4m3")
    a["k_scale"].fill_(scale)
    a["v_scale"].fill_(scale * 1.7)
    want = ref.compact(a, k, k, None, [0, 1024], None)
    kv.paged_compact_kv(k.cuda(), k.cuda(), None, [0, 1024], kv.PagedCache(**a))
    ref.assert_same_state(a, want)


def test_compact_bad_page_is_left_out():
    a = ref.make_cache(1, 1, 64, 8, 64, seed=2)
    k = torch.randn(64, 1, 64, generator=gen(1)).to(torch.bfloat16)
    want = ref.compact(a, k, k, None, [0, 64], None)
    hole = int(a["page_table"][0, 3])
    for name in ("k_pages", "v_pages", "pos", "weight"):
        want[name][hole] = a[name][hole].cpu()
    a["page_table"][0, 3] = 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.paged_compact_kv(k.cuda(), k.cuda(), None, [0, 64], kv.PagedCache(**a), status=status)
    ref.assert_same_state(a, want)
    with pytest.raises(kv.KvpopError):
        kv.check_status(status)


# ---------------------------------------------------------------- append

def check_append(a, cu, window, sinks, seed, fused=False, **kw):
    B, H = a["count"].shape
    d = a["k_pages"].shape[3]
    cu_ref = list(range(B + 1)) if cu is None else cu
    x = (3 * torch.randn(cu_ref[-1], (3 if fused else 1) * 2 * H, d, generator=gen(seed))).to(torch.bfloat16)
    k, v = x[:, -2 * H:-H], x[:, -H:]
    want, evicted = ref.append(a, k, v, cu_ref, window, sinks)
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    y = x.cuda()
    got = kv.paged_append_kv(y[:, -2 * H:-H] if fused else k.cuda(), y[:, -H:] if fused else v.cuda(), kv.PagedCache(**a),
                             window, sinks, cu_new=cu, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), evicted)
    ref.assert_same_state(a, want)


@pytest.mark.parametrize("B,H,d,page,cap,counts,window,sinks,dtype,layout", [
    (1, 1, 64, 8, 8, [[0]], 0, 0, "bf16", "hpd"),
    (2, 2, 64, 16, 100, [[100, 99], [0, 50]], 8, 4, "bf16", "hpd"),
    (3, 2, 128, 64, 300, [[300, 300], [-1, 300], [299, 400]], 32, 4, "bf16", "phd"),
    (2, 3, 128, 32, 500, [[500] * 3, [500, 0, -3]], 0, 0, "e4m3", "hpd"),
    (1, 2, 128, 16, 9000, [[9000, 8999]], 256, 4, "bf16", "hpd"),          # a cluster per row
    (60, 8, 64, 8, 40, [[40] * 8] * 60, 4, 2, "e4m3", "phd"),
])
def test_append_one(B, H, d, page, cap, counts, window, sinks, dtype, layout):
    a = ref.make_cache(B, H, d, page, cap, dtype, layout, seed=cap)
    fill_random(a, counts, seed=cap)
    for step in range(4):
        check_append(a, None, window, sinks, seed=step, fused=step % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_one_to_many_rows(dtype):
    """More rows than CTAs, each in several steps, full ones beside ones with room and ones that take no part."""
    B, H, cap = 150, 3, 4500
    counts = [[(cap, cap, cap - 1, 17, -1, 0, cap)[(b * H + h) % 7] for h in range(H)] for b in range(B)]
    a = ref.make_cache(B, H, 64, 64, cap, dtype, "phd", seed=cap)
    g = gen(3)
    page_count = a["pos"].shape[0]
    a["weight"].copy_(torch.randint(0, 500, (page_count, H, 64), generator=g).float())     # many equal weights
    a["pos"].copy_(torch.randint(0, 9000, (page_count, H, 64), generator=g).to(torch.int32))
    a["count"].copy_(torch.tensor(counts))
    a["seen"].fill_(9000)
    for name in ("k_pages", "v_pages"):
        a[name].view(torch.uint8).zero_()
    a["page_table"][5, 30] = -1                               # a hole in one full sequence
    before = a["page_table"].clone()
    a["page_table"][5, 30] = before[6, 0]                     # the reference: the hole's slots may not go
    hole = dict(a, page_table=a["page_table"].clone(), pos=a["pos"].clone())
    a["page_table"].copy_(before)
    x = torch.randn(B, 2 * H, 64, generator=g).to(torch.bfloat16)
    rows = [b for b in range(B) if b != 5]
    want, evicted = ref.append(hole, x[:, :H], x[:, H:], list(range(B + 1)), 256, 4)
    got = kv.paged_append_kv(x[:, :H].cuda().contiguous(), x[:, H:].cuda().contiguous(), kv.PagedCache(**a), 256, 4)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy()[rows], evicted[rows])
    for b in rows:
        t = before[b].long().cpu()
        for name in ("k_pages", "v_pages", "pos", "weight"):
            assert np.array_equal(ref.as_bytes(a[name].view(torch.uint8)[t] if a[name].dtype == ref.E4M3 else a[name][t]),
                                  ref.as_bytes(want[name].view(torch.uint8)[t] if a[name].dtype == ref.E4M3 else want[name][t])), (b, name)
    assert np.array_equal(a["count"].cpu().numpy(), want["count"].numpy())


@pytest.mark.parametrize("B,H,d,page,cap,counts,m,window,sinks,dtype", [
    (2, 2, 64, 16, 100, [[100, 90], [0, 97]], [8, 5], 8, 4, "bf16"),
    (3, 1, 128, 8, 64, [[64], [64], [10]], [32, 0, 32], 32, 4, "bf16"),
    (1, 2, 128, 64, 3000, [[3000, 2900]], [256], 256, 4, "e4m3"),
    (2, 2, 64, 32, 20000, [[20000, 19990], [5000, 20000]], [700, 650], 1000, 16, "bf16"),
    (1, 1, 64, 128, 131072, [[131072]], [300], 300, 4, "bf16"),                  # eight full slices
    (40, 4, 128, 16, 600, [[600] * 4] * 40, [17] * 40, 64, 4, "bf16"),
    (1, 3, 64, 8, 48, [[48, 47, -1]], [44], 44, 4, "e4m3"),                      # everything but the sinks may be recent
])
def test_append_chunk(B, H, d, page, cap, counts, m, window, sinks, dtype):
    a = ref.make_cache(B, H, d, page, cap, dtype, "hpd", seed=cap)
    fill_random(a, counts, seed=cap)
    cu = [0, *np.cumsum(m).tolist()]
    for step in range(2):
        check_append(a, cu, window, sinks, seed=step, fused=step == 1)


@pytest.mark.parametrize("chunk", [1, 5, 40])
def test_append_order_of_equal_and_odd_weights(chunk):
    """Ties go by position, NaN first of all, -0 with +0, infinities at the ends, all weights equal."""
    a = ref.make_cache(1, 4, 64, 16, 96, seed=5)
    fill_random(a, [[96] * 4], seed=5)
    pg, off = (x.cuda() for x in ref.slots_of(a, 0, 96, 16))
    odd = torch.tensor([0.0, -0.0, math.nan, -math.nan, math.inf, -math.inf, 1e-42, -1e-42, -1.0, 2.5]).cuda()
    a["weight"][pg, 0, off] = odd[torch.arange(96, device="cuda") % 10]
    a["weight"][pg, 1, off] = 1.25
    a["weight"][pg, 2, off] = torch.tensor([0.0, -0.0]).cuda()[torch.arange(96, device="cuda") % 2]
    a["weight"][pg, 3, off] = math.nan
    for step in range(3):
        check_append(a, None if chunk == 1 else [0, chunk], 40, 3, seed=step)


def test_append_reports_what_it_cannot_store():
    """Positions that leave nothing to evict, and a bad page: nothing is written there and the status says so."""
    a = ref.make_cache(1, 1, 64, 8, 16, seed=1)
    fill_random(a, [[16]], seed=1)
    pg, off = (x.cuda() for x in ref.slots_of(a, 0, 16, 8))
    a["pos"][pg, 0, off] = torch.arange(16, dtype=torch.int32, device="cuda") % 4          # all sinks
    for cu in (None, [0, 2]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        check_append(a, cu, 4, 4, seed=1, status=status)
        with pytest.raises(kv.KvpopError):
            kv.check_status(status)
    a = ref.make_cache(1, 1, 64, 8, 32, seed=1)
    fill_random(a, [[20]], seed=1)
    before = {n: ref.as_bytes(a[n]).copy() for n in ("k_pages", "v_pages", "pos", "weight")}
    a["page_table"][0, 2] = -4
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kv.paged_append_kv(k, k, kv.PagedCache(**a), 4, 4, status=status)
    assert got.tolist() == [[-2]] and int(a["count"]) == 21
    for n, x in before.items():
        assert np.array_equal(ref.as_bytes(a[n]), x)
    with pytest.raises(kv.KvpopError):
        kv.check_status(status)


def test_append_nothing():
    a = ref.make_cache(2, 1, 64, 8, 16, seed=1)
    fill_random(a, [[16], [3]], seed=1)
    check_append(a, [0, 0, 0], 4, 4, seed=1)
    check_append(a, [0, 0, 2], 4, 4, seed=1)


# ---------------------------------------------------------------- together

def serve(a, steps, window, sinks, G, seed, check=True):
    """Steps of decoding: append, attend, accumulate; each checked against the reference from the state before it."""
    B, H = a["count"].shape
    d = a["k_pages"].shape[3]
    for step in range(steps):
        check_append(a, None, window, sinks, seed=seed + step)
        q = (2 * torch.randn(B, H * G, d, generator=gen(seed + 100 + step))).to(torch.bfloat16).cuda()
        check_decode(a, q, 1 / math.sqrt(d), True)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_to_decoding(dtype):
    """Targets with window 0 (the attention a prompt's tokens have received), keep mask, compaction with those
    weights, then steps of append and attention that evict by them."""
    from future_attention_targets_b200.workloads import random_qk
    lens, Hkv, G, d, window, sinks, budget = (700, 333, 150), 2, 4, 128, 32, 4, 256
    T, cu = sum(lens), [0, *np.cumsum(lens).tolist()]
    qb, kb = random_qk(T, Hkv * G, Hkv, d, seed=11)
    dev = lambda bits: torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()
    q, k = dev(qb), dev(kb)
    v = torch.randn(T, Hkv, d, generator=gen(3)).to(torch.bfloat16).cuda()
    lse = kv.row_lse(q, k, cu)
    weight = kv.future_target(q, k, cu, 0, lse)
    keep = kv.keep_mask(weight, cu, window, sinks, [budget] * 3)
    a = ref.make_cache(3, Hkv, d, 64, budget, dtype, seed=3)
    want = ref.compact(a, k, v, keep, cu, weight)
    kv.paged_compact_kv(k, v, keep, cu, kv.PagedCache(**a), score=weight)
    ref.assert_same_state(a, want)
    assert a["count"].tolist() == [[256] * 2, [256] * 2, [150] * 2]
    serve(a, 5, window, sinks, G, seed=20)


def test_allocated_cache_grows_from_nothing():
    """PagedCache.allocate, token by token from an empty cache past its capacity."""
    cache = kv.PagedCache.allocate(2, 2, 64, capacity=20, page_size=8)
    a = dict(k_pages=cache.k_pages, v_pages=cache.v_pages, page_table=cache.page_table, count=cache.count, capacity=20,
             seen=cache.seen, pos=cache.pos, weight=cache.weight)
    serve(a, 26, 6, 2, 3, seed=50)
    assert cache.count.tolist() == [[20, 20]] * 2 and cache.seen.tolist() == [[26, 26]] * 2


def test_steps_in_a_graph():
    """A captured step replayed equals the same steps one by one; two graphs, each with a workspace of its own."""
    def fresh():
        a = ref.make_cache(3, 2, 128, 16, 200, seed=4)
        fill_random(a, [[200, 150], [200, 200], [0, 3]], seed=4)
        return a
    B, H, G, d = 3, 2, 4, 128
    x = torch.zeros(B, (G + 2) * H, d, dtype=torch.bfloat16, device="cuda")
    inputs = [torch.randn(x.shape, generator=gen(s)).to(torch.bfloat16).cuda() for s in range(8)]

    def step(cache, out, lse, ws, ev):
        kv.paged_append_kv(x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], cache, 16, 4, evicted=ev)
        kv.paged_decode_attention(x[:, :G * H], cache, accumulate=True, out=out, lse=lse, workspace=ws)

    def buffers(cache):
        return (torch.empty(B, G * H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, G * H, device="cuda"),
                torch.empty(kv.paged_decode_workspace_bytes(cache, G * H), dtype=torch.uint8, device="cuda"),
                torch.empty(B, H, dtype=torch.int32, device="cuda"))

    eager = fresh()
    ec = kv.PagedCache(**eager)
    eb = buffers(ec)
    graphs = []
    for _ in range(2):
        a = fresh()
        c = kv.PagedCache(**a)
        bufs = buffers(c)
        saved = {n: a[n].clone() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(c, *bufs)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(c, *bufs)
        for n, t in saved.items():
            a[n].copy_(t)
        graphs.append((graph, a, bufs))
    for inp in inputs:
        x.copy_(inp)
        step(ec, *eb)
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, a, bufs in graphs:
            assert torch.equal(bufs[0], eb[0]) and torch.equal(bufs[1], eb[1]) and torch.equal(bufs[3], eb[3])
    state = {n: eager[n].cpu() for n in ("k_pages", "v_pages", "pos", "weight", "count", "seen")}
    for _, a, _ in graphs:
        ref.assert_same_state(a, state)
