"""Performance cases of the paged key-value cache: filling it from a prompt, appending tokens to it with
eviction by accumulated attention weight, and one decode step of attention over it.

A cache row is (sequence b, KV head h).  Its slots 0 .. count - 1 lie in pages of `page` slots: slot c of row
(b, h) is [table[b, c // page], h, c % page] of the pools k, v [N, H, page, d], pos and weight [N, H, page].
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
SCALE_K, SCALE_V = 0.02, 0.015        # e4m3 caches: scale of KV head 0; head h has (1 + h / 8) times it
NEVER = 2**63 - 1


def listed():
    return [
        # One step of a small model's tests: a handful of tokens, ragged, GQA 2.  Latency only.
        dict(name="decode small", op="decode", batch=2, q_heads=4, kv_heads=2, d=64, page=16, cap=200, fill="ragged",
             dtype="bf16", layout="hpd", weight=True, fused=False),
        # One conversation on an 8B-class layer at the budget of 4 + 3,772 + 256 entries per head.
        dict(name="decode one", op="decode", batch=1, q_heads=32, kv_heads=8, d=128, page=64, cap=4032, fill="full",
             dtype="bf16", layout="hpd", weight=True, fused=True),
        # A serving batch in steady state: every row at its budget, weights accumulated for the eviction.
        dict(name="decode batch", op="decode", batch=64, q_heads=32, kv_heads=8, d=128, page=64, cap=4032, fill="full",
             dtype="bf16", layout="hpd", weight=True, fused=True),
        # A dense cache of very different lengths, some empty, 5 query heads per KV head, token-major pages of 16.
        dict(name="decode ragged", op="decode", batch=40, q_heads=40, kv_heads=8, d=128, page=16, cap=16384,
             fill="ragged", dtype="bf16", layout="phd", weight=False, fused=False),
        # A few very long contexts without eviction.
        dict(name="decode long", op="decode", batch=4, q_heads=32, kv_heads=8, d=128, page=128, cap=131071, fill="full",
             dtype="bf16", layout="hpd", weight=False, fused=False),
        # A large batch over an 8-bit cache, 7 query heads per KV head.
        dict(name="decode e4m3", op="decode", batch=96, q_heads=28, kv_heads=4, d=128, page=32, cap=8192, fill="full",
             dtype="e4m3", layout="hpd", weight=True, fused=True),
        # The steady state of one conversation: one token in, the least attended one out.
        dict(name="append one", op="append", batch=1, kv_heads=8, d=128, page=64, cap=4032, window=256, sinks=4, new=1,
             fill="full", dtype="bf16", layout="hpd", fused=True),
        # The same for a large serving batch.
        dict(name="append batch", op="append", batch=256, kv_heads=8, d=128, page=64, cap=4032, window=256, sinks=4,
             new=1, fill="full", dtype="bf16", layout="hpd", fused=True),
        # Chunks of a prompt (up to 256 tokens, of different lengths) into caches that are full or nearly so.
        dict(name="append chunk", op="append", batch=24, kv_heads=8, d=128, page=16, cap=16000, window=256, sinks=4,
             new=256, fill="ragged", dtype="e4m3", layout="phd", fused=False),
        # A short prompt, dense.
        dict(name="compact short", op="compact", batch=3, kv_heads=2, d=64, page=16, tokens=300, cap=300, window=16,
             sinks=4, dtype="bf16", layout="hpd"),
        # The 16,384-token prompt cut to its budget.
        dict(name="compact prompt", op="compact", batch=1, kv_heads=8, d=128, page=64, tokens=16384, cap=4032,
             window=256, sinks=4, dtype="bf16", layout="hpd"),
        # Eight packed prompts of different lengths into an 8-bit cache.
        dict(name="compact packed", op="compact", batch=8, kv_heads=8, d=128, page=32, tokens=100003, cap=8192,
             window=256, sinks=4, dtype="e4m3", layout="phd"),
    ]


def draw(rng):
    spread = lambda lo, hi: min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))
    op = rng.choice(["decode", "decode", "append", "compact"])
    d = rng.choice([64, 128, 128])
    case = dict(op=op, d=d, page=rng.choice([8, 16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "e4m3"]),
                layout=rng.choice(["hpd", "hpd", "phd"]))
    heads = rng.choice([1, 2, 4, 5, 8, 8, 16])
    if op == "compact":
        tokens = spread(100, 131072)
        batch = spread(1, min(64, max(1, tokens // 50)))
        cap = max(64, spread(max(1, tokens // batch // 8), max(1, 2 * tokens // batch)))
        return dict(case, batch=batch, kv_heads=min(heads, 8), tokens=tokens, cap=cap, window=min(256, cap // 4), sinks=4)
    cap = spread(64, 131072)
    fill = rng.choice(["full", "ragged"])
    if op == "decode":
        group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
        batch = spread(1, max(1, min(256, 4 * 32 * 131072 // (cap * heads * max(4, group)))))
        return dict(case, batch=batch, q_heads=heads * group, kv_heads=heads, cap=cap, fill=fill,
                    weight=rng.random() < 0.5, fused=rng.random() < 0.5)
    batch = spread(1, max(1, min(256, 256 * 8 * 4032 // (cap * heads))))
    window = min(256, cap // 4)
    new = 1 if rng.random() < 0.5 else spread(1, window)
    return dict(case, batch=batch, kv_heads=heads, cap=cap, window=window, sinks=4, new=new, fill=fill,
                fused=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lengths(case, gen):
    """Tokens seen by each sequence [B]: full rows have seen up to four times their capacity; ragged ones are
    spread over the lengths from one token up (the first is the longest, one in sixteen is empty when it is
    only read)."""
    B, cap = case["batch"], case["cap"]
    u = torch.rand(B, generator=gen, device="cuda", dtype=torch.float64)
    if case["fill"] == "full":
        return cap + (u * 3 * cap).long()
    if case["op"] == "append":
        return cap - case["new"] + (u * 2 * case["new"]).long()
    n = torch.exp(u * math.log(cap)).long().clamp_(1, cap)
    n[torch.arange(B, device="cuda") % 16 == 15] = 0
    n[0] = cap
    return n


def _pools(case, gen, n_pages):
    """The two pools in bf16 or e4m3, as an allocator would hand them out: used pages and old content alike."""
    H, P, d = case["kv_heads"], case["page"], case["d"]
    pools = []
    for spread in (SCALE_K, SCALE_V):
        x = torch.empty((n_pages, H, P, d) if case["layout"] == "hpd" else (n_pages, P, H, d), device="cuda",
                        dtype=torch.bfloat16).normal_(generator=gen)
        if case["dtype"] == "e4m3":
            x = x.div_(spread).to(E4M3)
        pools.append(x if case["layout"] == "hpd" else x.permute(0, 2, 1, 3))
    return pools


def _table(case, gen, slots):
    """Page table [B, max_pages] for rows of `slots` [B] slots, pages in no order; -1 where none is needed."""
    B, P = case["batch"], case["page"]
    max_pages = -(-case["cap"] // P)
    n_pages = B * max_pages + 3
    table = torch.randperm(n_pages, generator=gen, device="cuda")[: B * max_pages].view(B, max_pages).to(torch.int32)
    need = torch.arange(max_pages, device="cuda")[None, :] * P < slots[:, None]
    return torch.where(need, table, -1).to(torch.int32).contiguous(), n_pages


def _rows(state, slots):
    """Index (page, head, offset) of slots [B, H, n] in the pools."""
    B, H = slots.shape[:2]
    P = state["page"]
    table = state["table"].clamp(min=0).long()
    page = table[torch.arange(B, device="cuda")[:, None, None], slots // P]
    return page, torch.arange(H, device="cuda")[None, :, None].expand_as(slots), slots % P


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    H, P, d, B = case["kv_heads"], case["page"], case["d"], case["batch"]
    state = dict(case=case, page=P, cap=case["cap"])
    head = 1 + torch.arange(H, device="cuda", dtype=torch.float32) / 8
    state["k_scale"], state["v_scale"] = (SCALE_K * head, SCALE_V * head) if case["dtype"] == "e4m3" else (None, None)
    if case["op"] == "compact":
        return _prepare_compact(case, gen, state)
    L = _lengths(case, gen)
    n = L.clamp(max=case["cap"])
    state["table"], n_pages = _table(case, gen, n if case["op"] == "decode" else torch.full_like(n, case["cap"]))
    state["k"], state["v"] = _pools(case, gen, n_pages)
    state["count"] = n.to(torch.int32)[:, None].repeat(1, H)
    state["seen"] = L.to(torch.int32)[:, None].repeat(1, H)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    # Accumulated weights: heavy-tailed, one in a hundred never attended.
    weight = torch.exp(2 * normal(n_pages, H, P))
    weight[torch.rand((n_pages, H, P), generator=gen, device="cuda") < 0.01] = 0
    state["weight"] = weight
    if case["op"] == "decode":
        if not case["weight"]:
            state["weight"] = None
        state["pos"] = None
        Hq = case["q_heads"]
        state["scale"] = 1 / math.sqrt(d)
        wide = (2 * normal(B, Hq + (2 * H if case["fused"] else 0), d)).to(torch.bfloat16)   # q, or q of q | k | v
        state["q"] = wide[:, :Hq]
        return state
    # Positions in the slots: sinks, a spread choice of the middle and the recent window, in no order (evictions
    # have scattered them); all positions in order where nothing was evicted yet.
    S, W, C = case["sinks"], case["window"], case["cap"]
    c = torch.arange(C, device="cuda")[None, None, :]
    Lr, nr = L[:, None, None], n[:, None, None]
    ratio = (Lr - W - S).double() / (nr - W - S).clamp(min=1)
    jitter = torch.rand((B, H, C), generator=gen, device="cuda") * ratio.floor().clamp(min=1)
    middle = S + torch.floor((c - S) * ratio).long() + jitter.long()
    pos = torch.where(c < S, c, torch.where(c >= nr - W, Lr - (nr - c), middle))
    pos = torch.where(Lr > nr, pos, c.expand_as(pos))
    order = torch.rand((B, H, C), generator=gen, device="cuda")
    order = torch.where((c < nr) & (Lr > nr), order, 2.0 + c).argsort(dim=2)
    pos = torch.gather(pos, 2, order).to(torch.int32)
    state["pos"] = torch.full((n_pages, H, P), -1, dtype=torch.int32, device="cuda")
    state["pos"][_rows(state, c.expand(B, H, C))] = pos
    # New tokens: one per sequence, or chunks of up to `new` of them (the first whole, the others 0 .. new; the case
    # alone sets the lengths, the seed only the values).
    if case["new"] == 1:
        m = torch.ones(B, dtype=torch.long)
    else:
        m = torch.randint(0, case["new"] + 1, (B,), generator=torch.Generator().manual_seed(B * case["new"]))
        m[0] = case["new"]
    cu = [0] + torch.cumsum(m, 0).tolist()
    state["cu_new"] = None if case["new"] == 1 else cu
    state["m"] = m.cuda()
    state["m_max"] = int(m.max())
    state["token_seq"] = torch.repeat_interleave(torch.arange(B), m).cuda()
    state["token_at"] = (torch.arange(cu[-1]) - torch.tensor(cu[:-1]).repeat_interleave(m)).cuda()
    wide = normal(cu[-1], (6 if case["fused"] else 2) * H, d).to(torch.bfloat16)
    state["k_new"], state["v_new"] = wide[:, -2 * H:-H], wide[:, -H:]
    state["window"], state["sinks"] = W, S
    return state


def _prepare_compact(case, gen, state):
    H, B, T, S, W = case["kv_heads"], case["batch"], case["tokens"], case["sinks"], case["window"]
    cuts = torch.rand(B, generator=gen, device="cuda").add_(0.15).cumsum(0)
    ends = (cuts / cuts[-1] * T).long().cpu().tolist()
    cu = [0] + ends[:-1] + [T]
    score = torch.exp(2 * torch.randn((H, T), generator=gen, device="cuda"))   # heavy-tailed attention mass
    keep = torch.zeros((H, T), dtype=torch.uint8, device="cuda")
    for b in range(B):
        lo, hi = cu[b], cu[b + 1]
        if hi - lo <= case["cap"]:
            keep[:, lo:hi] = 1
            continue
        keep[:, lo:lo + S] = 1
        keep[:, hi - W:hi] = 1
        top = score[:, lo + S:hi - W].topk(case["cap"] - S - W, dim=1).indices
        keep[:, lo + S:hi - W].scatter_(1, top, 1)
    state["table"], n_pages = _table(case, gen, torch.full((B,), case["cap"], device="cuda"))
    state["k"], state["v"] = _pools(case, gen, n_pages)
    state["pos"] = torch.full((n_pages, H, case["page"]), -1, dtype=torch.int32, device="cuda")
    state["weight"] = torch.zeros((n_pages, H, case["page"]), device="cuda")
    state["count"] = torch.zeros((B, H), dtype=torch.int32, device="cuda")
    state["seen"] = torch.zeros((B, H), dtype=torch.int32, device="cuda")
    state["cu"] = cu
    length = torch.tensor(cu[1:]) - torch.tensor(cu[:-1])
    state["length"] = length.cuda()
    state["token_seq"] = torch.repeat_interleave(torch.arange(B), length).cuda()
    state["start"] = torch.tensor(cu[:-1]).cuda()
    state["score"], state["keep"] = score, keep
    state["k_in"], state["v_in"] = (torch.randn((T, H, case["d"]), generator=gen, device="cuda").to(torch.bfloat16)
                                    for _ in range(2))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    return {"decode": _decode, "append": _append, "compact": _compact}[op](state)


def _run_own(op, state):
    import future_attention_targets_b200 as kv
    if "cache" not in state:          # the handle that a serving program makes once, with its output buffers
        state["cache"] = kv.PagedCache(state["k"], state["v"], state["table"], state["count"], capacity=state["cap"],
                                       seen=state["seen"], pos=state["pos"], weight=state["weight"],
                                       k_scale=state["k_scale"], v_scale=state["v_scale"])
        if op == "decode":
            B, Hq, _ = state["q"].shape
            state["out"] = torch.empty_like(state["q"], memory_format=torch.contiguous_format)
            state["lse"] = torch.empty((B, Hq), device="cuda")
            need = kv.paged_decode_workspace_bytes(state["cache"], Hq)
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if op == "decode":
        out, lse = kv.paged_decode_attention(state["q"], state["cache"], scale=state["scale"],
                                             accumulate=state["weight"] is not None, out=state["out"],
                                             lse=state["lse"], workspace=state["workspace"])
        return {"out": out, "lse": lse} if state["weight"] is None else {"out": out, "lse": lse, "weight": state["weight"]}
    if op == "append":
        evicted = kv.paged_append_kv(state["k_new"], state["v_new"], state["cache"], state["window"], state["sinks"],
                                     cu_new=state["cu_new"])
        return dict(_cache_state(state), evicted=evicted)
    kv.paged_compact_kv(state["k_in"], state["v_in"], state["keep"], state["cu"], state["cache"], score=state["score"])
    return _cache_state(state)


def _cache_state(state):
    return {name: state[name] for name in ("k", "v", "pos", "weight", "count", "seen")}


def _gather(pool, index):
    if pool.dtype == E4M3:
        return pool.view(torch.uint8)[index].view(E4M3).float()
    return pool[index].float()


def _put(pool, index, rows, scale):
    """Rows [tokens, H, d] into the pool; an 8-bit pool holds them over the head's scale, clipped to its range."""
    if pool.dtype == E4M3:
        rows = (rows.float() / scale[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        pool = pool.view(torch.uint8)
    pool[index] = rows


def _decode(state):
    B, Hq, d = state["q"].shape
    H, C = state["count"].shape[1], state["cap"]
    slots = torch.arange(C, device="cuda")
    index = _rows(state, slots.expand(B, H, C))
    valid = (slots < state["count"][:, :, None].clamp(max=C))[:, :, None, :]
    q = state["q"].float().reshape(B, H, Hq // H, d)
    s = q @ _gather(state["k"], index).transpose(2, 3) * state["scale"]
    if state["k_scale"] is not None:
        s = s * state["k_scale"][:, None, None]
    s = s.masked_fill(~valid, -math.inf)
    top = s.amax(3, keepdim=True).clamp(min=-3e38)
    e = torch.exp(s - top)
    total = e.sum(3, keepdim=True)
    p = e / total.clamp(min=1e-38)
    out = p @ _gather(state["v"], index).masked_fill(~valid.transpose(2, 3), 0)
    if state["v_scale"] is not None:
        out = out * state["v_scale"][:, None, None]
    got = {"out": out.reshape(B, Hq, d).to(torch.bfloat16), "lse": (top + torch.log(total)).reshape(B, Hq)}
    if state["weight"] is not None:
        # Slots past the count point at page 0 or at another's old slot: they add nothing.
        state["weight"].index_put_(index, p.sum(2), accumulate=True)
        got["weight"] = state["weight"]
    return got


def _append(state):
    count, seen, cap = state["count"].long(), state["seen"].long(), state["cap"]
    B, H = count.shape
    S, W, m, m_max = state["sinks"], state["window"], state["m"][:, None], state["m_max"]
    n = count.clamp(max=cap)
    slots = torch.arange(cap, device="cuda").expand(B, H, cap)
    index = _rows(state, slots)
    weight, pos = state["weight"][index], state["pos"][index].long()
    # Eviction order: the least weight first (NaN below every number, -0 equal to +0), of equal ones the latest.
    bits = (weight + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(2**31) - 1 - bits)
    key = torch.where(weight.isnan(), -(2**31), key) * 2**32 + (2**31 - 1 - pos)
    may_go = (slots < n[:, :, None]) & (pos >= S) & (pos < (seen + m - W)[:, :, None])
    least, victim = torch.where(may_go, key, NEVER).topk(m_max, dim=2, largest=False, sorted=True)
    free = torch.minimum(m, cap - n)
    taken = (torch.arange(m_max, device="cuda") < (m - free)[:, :, None]) & (least < NEVER)
    victim = torch.where(taken, victim, cap).sort(dim=2).values
    # The i-th new token of a sequence goes to slot n + i while there is room, then to the victims in slot order.
    b, i = state["token_seq"], state["token_at"][:, None]
    free_t = free[b]
    at_victim = victim[b[:, None], torch.arange(H, device="cuda"), (i - free_t).clamp(min=0)]
    slot = torch.where(i < free_t, n[b] + i, at_victim)
    page = state["table"].long()[b[:, None], slot // state["page"]]
    index = (page, torch.arange(H, device="cuda").expand_as(page), slot % state["page"])
    evicted = torch.where(i < free_t, -1, state["pos"][index])
    _put(state["k"], index, state["k_new"], state["k_scale"])
    _put(state["v"], index, state["v_new"], state["v_scale"])
    state["pos"][index] = (seen[b] + i).to(torch.int32)
    state["weight"][index] = 0.0
    state["count"].copy_((n + m).clamp(max=cap))
    state["seen"].copy_(seen + m)
    return dict(_cache_state(state), evicted=evicted.to(torch.int32))


def _compact(state):
    keep, cap, start = state["keep"] != 0, state["cap"], state["start"]
    H, T = keep.shape
    before = torch.cat([torch.zeros((H, 1), dtype=torch.long, device="cuda"), keep.long().cumsum(1)], 1)
    slot = before[:, :-1] - before[:, start][:, state["token_seq"]]
    h, t = (keep & (slot < cap)).nonzero(as_tuple=True)
    slot, b = slot[h, t], state["token_seq"][t]
    index = (state["table"].long()[b, slot // state["page"]], h, slot % state["page"])
    for pool, rows, scale in ((state["k"], state["k_in"], state["k_scale"]), (state["v"], state["v_in"], state["v_scale"])):
        _put(pool, index, rows[t, h], None if scale is None else scale[h])
    state["pos"][index] = (t - start[b]).to(torch.int32)
    state["weight"][index] = state["score"][h, t]
    total = before[:, start + state["length"]] - before[:, start]
    state["count"].copy_(total.T.clamp(max=cap))
    state["seen"].copy_(state["length"][:, None].expand(-1, H))
    return _cache_state(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, d, cap, B = case["kv_heads"], case["d"], case["cap"], case["batch"]
    elt = 1 if case["dtype"] == "e4m3" else 2
    if case["op"] == "decode":
        # Ragged lengths are spread over the logarithm from 1 to cap: (cap - 1) / ln cap on average.
        slots = H * (B * cap if case["fill"] == "full" else cap + (B - 1) * (cap - 1) / math.log(cap) * 15 / 16)
        rows = B * case["q_heads"] * (4 * d + 4)                        # q and out in bf16, lse
        return {"bytes": slots * (2 * d * elt + (8 if case["weight"] else 0)) + rows,
                "flops": 4.0 * slots * d * case["q_heads"] / H}
    if case["op"] == "append":
        tokens = B if case["new"] == 1 else case["new"] + (B - 1) * case["new"] / 2
        looked = B * H * cap                                            # weight and position of every slot
        return {"bytes": looked * 8 + tokens * H * (2 * d * (2 + elt) + 12) + 16 * B * H, "flops": looked}
    kept = H * min(case["tokens"], B * cap)
    return {"bytes": H * case["tokens"] + kept * (2 * d * (2 + elt) + 12) + 8 * B * H, "flops": kept}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "compact": _exact_compact}[case["op"]](state)


def _exact_decode(state):
    """Row by row: the scores, their exponentials over the largest and the weighted sum, in float64."""
    q = state["q"].double()
    B, Hq, d = q.shape
    H, P = state["count"].shape[1], state["page"]
    G = Hq // H
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    weight = None if state["weight"] is None else state["weight"].double()
    counts, table = state["count"].tolist(), state["table"].tolist()
    for b in range(B):
        for h in range(H):
            n = min(counts[b][h], state["cap"])
            if n <= 0:
                continue
            pages = torch.tensor(table[b][: -(-n // P)], device="cuda")
            k = state["k"][:, h].view(torch.uint8)[pages].view(state["k"].dtype).double().reshape(-1, d)[:n]
            v = state["v"][:, h].view(torch.uint8)[pages].view(state["v"].dtype).double().reshape(-1, d)[:n]
            if state["k_scale"] is not None:
                k, v = k * state["k_scale"][h].double(), v * state["v_scale"][h].double()
            g = slice(h * G, (h + 1) * G)
            x = (q[b, g] @ k.T) * state["scale"]
            lse[b, g] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, g, None])
            out[b, g] = p @ v
            if weight is not None:
                add = torch.zeros(len(pages) * P, dtype=torch.float64, device="cuda")
                add[:n] = p.sum(0)
                weight[pages, h] += add.view(-1, P)
    got = {"out": out, "lse": lse}
    return got if weight is None else dict(got, weight=weight)


def _quotient(rows, scale, pool):
    """What a pool's slot stands for before its rounding: the row itself, or the row over its head's scale."""
    rows = rows.double()
    return rows if pool.dtype != E4M3 else (rows / scale.double()[:, None]).clamp(-448, 448)


def _exact_append(state):
    """Row by row on the host: the free slots, then the slots in eviction order, found by sorting tuples."""
    counts, seens, table = state["count"].tolist(), state["seen"].tolist(), state["table"].tolist()
    B, H, P, cap, S, W = len(counts), len(counts[0]), state["page"], state["cap"], state["sinks"], state["window"]
    if B * H * cap > 9_000_000:
        return None
    weights, positions = state["weight"].cpu().numpy(), state["pos"].cpu().numpy()
    k, v, weight = state["k"].double(), state["v"].double(), state["weight"].double()
    cu = state["cu_new"] or list(range(B + 1))
    token, head, page, offset = [], [], [], []
    for b in range(B):
        m = cu[b + 1] - cu[b]
        for h in range(H):
            n = min(counts[b][h], cap)
            w, x = weights[table[b], h].reshape(-1)[:n], positions[table[b], h].reshape(-1)[:n]
            may_go = ((x >= S) & (x < seens[b][h] + m - W)).nonzero()[0]
            need = max(0, m - (cap - n))
            if need:
                low = may_go[w[may_go] <= sorted(w[may_go].tolist())[need - 1]].tolist()
                low = sorted(low, key=lambda c: (w[c], -x[c]))[:need]
            else:
                low = []
            to = list(range(n, min(cap, n + m))) + sorted(low)
            token += range(cu[b], cu[b] + m)
            head += [h] * m
            page += [table[b][c // P] for c in to]
            offset += [c % P for c in to]
    token, index = torch.tensor(token, device="cuda"), tuple(torch.tensor(x, device="cuda") for x in (head, page, offset))
    index = (index[1], index[0], index[2])
    heads = index[1]
    k[index] = _quotient(state["k_new"], state["k_scale"], state["k"])[token, heads]
    v[index] = _quotient(state["v_new"], state["v_scale"], state["v"])[token, heads]
    weight[index] = 0
    return {"k": k, "v": v, "pos": None, "weight": weight, "count": None, "seen": None, "evicted": None}


def _exact_compact(state):
    """Row by row: the first `cap` kept positions of each sequence and head, in order."""
    k, v, weight = state["k"].double(), state["v"].double(), state["weight"].double()
    k_in = _quotient(state["k_in"], state["k_scale"], state["k"])
    v_in = _quotient(state["v_in"], state["v_scale"], state["v"])
    P, cu, table = state["page"], state["cu"], state["table"].long()
    for b in range(len(cu) - 1):
        for h in range(state["keep"].shape[0]):
            at = state["keep"][h, cu[b]:cu[b + 1]].nonzero()[:, 0][: state["cap"]] + cu[b]
            slot = torch.arange(len(at), device="cuda")
            page, offset = table[b, slot // P], slot % P
            k[page, h, offset], v[page, h, offset] = k_in[at, h], v_in[at, h]
            weight[page, h, offset] = state["score"][h, at].double()
    return {"k": k, "v": v, "pos": None, "weight": weight, "count": None, "seen": None}
