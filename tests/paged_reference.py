"""Plain 64-bit reference of the paged cache on the CPU: dictionaries of rows, loops and numpy, nothing shared
with the kernels."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
EPS32 = 2.0 ** -24            # half a step of fp32
HALF_BF16 = 2.0 ** -8         # half a step of bf16, relative


def make_cache(B, Hkv, d, page, cap, dtype="bf16", layout="hpd", seed=0, spare=3, weight=True, poison=True, device="cuda"):
    """Pools full of NaN (where poison), a shuffled page table, empty rows.  Returns the PagedCache arguments."""
    g = torch.Generator().manual_seed(seed)
    max_pages = -(-cap // page)
    N = B * max_pages + spare
    dt = E4M3 if dtype == "e4m3" else torch.bfloat16
    pools = []
    for _ in range(2):
        x = torch.full((N, Hkv, page, d) if layout == "hpd" else (N, page, Hkv, d), float("nan") if poison else 0.0)
        x = x.to(dt).to(device)
        pools.append(x if layout == "hpd" else x.permute(0, 2, 1, 3))
    table = torch.randperm(N, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32).to(device)
    a = dict(k_pages=pools[0], v_pages=pools[1], page_table=table,
             count=torch.zeros(B, Hkv, dtype=torch.int32, device=device), capacity=cap,
             seen=torch.zeros(B, Hkv, dtype=torch.int32, device=device),
             pos=torch.full((N, Hkv, page), -7, dtype=torch.int32, device=device))
    if weight:
        a["weight"] = torch.full((N, Hkv, page), float("nan") if poison else 0.0, device=device)
    if dtype == "e4m3":
        a["k_scale"] = (0.02 * (1 + torch.arange(Hkv) / 8)).float().to(device)
        a["v_scale"] = (0.015 * (1 + torch.arange(Hkv) / 4)).float().to(device)
    return a


def slots_of(a, b, n, page):
    """(pages, offsets) of slots 0 .. n - 1 of sequence b."""
    c = torch.arange(n)
    return a["page_table"][b].cpu().long()[c // page], c % page


def as_bytes(t):
    """Bit patterns, for comparisons that count NaN as equal to itself; an e4m3 NaN has no sign (conversions
    give 0x7f or 0xff for the same NaN)."""
    if t.dtype == E4M3:
        x = t.cpu().contiguous().view(torch.uint8).numpy()
        return np.where((x & 0x7F) == 0x7F, 0x7F, x)
    return t.cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.uint8 if t.element_size() == 1
                                     else torch.int32).numpy()


def set_rows(a, b, h, k_rows, v_rows, pos=None, weight=None):
    """Puts rows [n, d] (fp32 values that the pool's type holds, times the scale) into slots 0 .. n - 1."""
    n, page = k_rows.shape[0], a["k_pages"].shape[2]
    pg, off = (x.to(a["k_pages"].device) for x in slots_of(a, b, n, page))
    for pool, rows in ((a["k_pages"], k_rows), (a["v_pages"], v_rows)):
        if pool.dtype == E4M3:
            pool.view(torch.uint8)[pg, h, off] = rows.to(E4M3).view(torch.uint8).to(pool.device)
        else:
            pool[pg, h, off] = rows.to(pool.dtype).to(pool.device)
    if pos is not None:
        a["pos"][pg, h, off] = torch.as_tensor(pos, dtype=torch.int32).to(pool.device)
    if weight is not None:
        a["weight"][pg, h, off] = torch.as_tensor(weight, dtype=torch.float32).to(pool.device)


def get_rows(a, b, h, n):
    """K, V rows [n, d] in float64, scales applied."""
    page = a["k_pages"].shape[2]
    pg, off = (x.to(a["k_pages"].device) for x in slots_of(a, b, n, page))
    got = []
    for pool, scale in (("k_pages", "k_scale"), ("v_pages", "v_scale")):
        t = a[pool]
        t = t.view(torch.uint8)[pg, h, off].view(E4M3) if t.dtype == E4M3 else t[pg, h, off]
        x = t.float().cpu().double().numpy()
        if a.get(scale) is not None:
            x = x * float(a[scale][h].double())
        got.append(x)
    return got


def decode(q, a, scale, bad=()):
    """out, lse, and per (b, h) the weights to add, with the bounds of section "tolerances" below; `bad`: pages
    (b, entry) whose slots take no part."""
    B, Hq, d = q.shape
    Hkv, page, cap = a["count"].shape[1], a["k_pages"].shape[2], a["capacity"]
    G = Hq // Hkv
    q = q.detach().float().cpu().double().numpy()
    out, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -math.inf)
    tol_out, tol_lse = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    add = {}
    eight = a["k_pages"].dtype == E4M3
    for b in range(B):
        for h in range(Hkv):
            n = min(max(int(a["count"][b, h]), 0), cap)
            use = np.array([c for c in range(n) if (b, c // page) not in bad], dtype=int)
            if not len(use):
                continue
            k, v = (x[use] for x in get_rows_skipping(a, b, h, n, bad, page))
            for g in range(h * G, (h + 1) * G):
                s = k @ q[b, g] * scale
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                out[b, g] = p @ v
                lse[b, g] = top + math.log(e.sum())
                # Tolerances.  A score sums d products in fp32, in any order and with truncation (2 EPS32 a step):
                # off by at most d * 2 EPS32 * sum |q k| scale, plus 3 roundings of the result.  An 8-bit cache's
                # fp16 q is off by 2^-25 of the row's largest entry at most.
                size = (np.abs(k) @ np.abs(q[b, g])).max() * scale
                err = d * 2 * EPS32 * size + 6 * EPS32 * np.abs(s).max()
                if eight:
                    err += 2.0 ** -25 * np.abs(q[b, g]).max() * np.abs(k).sum(1).max() * scale
                # exp2: 2^-22 relative, its argument 2 roundings of up to |s - lse| in log2 units; sums of n terms
                # run over 16-slot steps, warps and splits: n / 16 + 40 additions at most.
                err += 2.0 ** -22 + 4 * EPS32 * np.abs(s - lse[b, g]).max() * 1.5
                steps = (n / 16 + 40) * 2 * EPS32
                tol_lse[b, g] = err + steps + 4 * EPS32 * (1 + abs(lse[b, g]) + np.abs(s).max())
                # Numerator and denominator each off by err + steps; p enters the product as two parts (2^-17).
                rel = 2 * (err + steps) + 2.0 ** -17
                tol_out[b, g] = HALF_BF16 * np.abs(out[b, g]) * (1 + rel) + rel * (p @ np.abs(v)) + 1e-30
                w = add.setdefault((b, h), [np.zeros(n), np.zeros(n)])
                w[0][use] += p
                w[1][use] += p * (2 * (err + steps) + (G + 2) * 2 * EPS32) + 1e-37
    return out, lse, tol_out, tol_lse, add


def get_rows_skipping(a, b, h, n, bad, page):
    """get_rows with the bad pages' slots as zeros (they are not looked up)."""
    if not bad:
        return get_rows(a, b, h, n)
    c = dict(a)
    c["page_table"] = a["page_table"].clone()
    for (bb, e) in bad:
        c["page_table"][bb, e] = 0
    return get_rows(c, b, h, n)


def quantise(x, pool_dtype, scale):
    """bf16 rows as the pool holds them."""
    if pool_dtype != E4M3:
        return x
    # The fp32 quotient is IEEE in numpy; clip keeps NaN.
    with np.errstate(all="ignore"):
        y = np.clip((x.float().numpy() / np.float32(scale)).astype(np.float32), -448, 448)
    return torch.from_numpy(y).to(E4M3)


def append(a, k_new, v_new, cu, window, sinks):
    """The state after appending, as a copy of the arguments on the CPU, and evicted [T_new, Hkv]."""
    st = {k: (v.detach().cpu().clone() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    B, H = st["count"].shape
    page, cap = st["k_pages"].shape[2], st["capacity"]
    T = cu[-1]
    evicted = np.full((T, H), -2, dtype=np.int32)
    for b in range(B):
        m = cu[b + 1] - cu[b]
        if m == 0:
            continue
        for h in range(H):
            n = int(st["count"][b, h])
            if n < 0:
                continue
            n = min(n, cap)
            seen = int(st["seen"][b, h])
            pg, off = slots_of(st, b, cap, page)
            w = st["weight"][pg, h, off].double().numpy()
            x = st["pos"][pg, h, off].long().numpy()
            to = list(range(n, min(cap, n + m)))
            out = [-1] * len(to)
            may = [c for c in range(n) if x[c] >= sinks and x[c] < seen + m - window]
            may.sort(key=lambda c: (0, -x[c]) if math.isnan(w[c]) else (1, w[c], -x[c]))
            victims = sorted(may[:m - len(to)])
            out += [int(x[c]) for c in victims]
            to += victims
            for i, c in enumerate(to):
                t = cu[b] + i
                P, o = int(pg[c]), int(off[c])
                for pool, src, sc in (("k_pages", k_new, "k_scale"), ("v_pages", v_new, "v_scale")):
                    row = src[t, h].cpu()
                    if st[pool].dtype == E4M3:
                        st[pool].view(torch.uint8)[P, h, o] = quantise(row, E4M3, float(st[sc][h]) if st.get(sc) is not None else 1.0).view(torch.uint8)
                    else:
                        st[pool][P, h, o] = row
                st["pos"][P, h, o] = seen + i
                st["weight"][P, h, o] = 0.0
                evicted[t, h] = out[i]
            st["count"][b, h] = min(n + m, cap)
            st["seen"][b, h] = seen + m
    return st, evicted


def compact(a, k, v, keep, cu, score):
    st = {x: (y.detach().cpu().clone() if isinstance(y, torch.Tensor) else y) for x, y in a.items()}
    B, H = st["count"].shape
    page, cap = st["k_pages"].shape[2], st["capacity"]
    k, v = k.cpu(), v.cpu()
    for b in range(B):
        L = cu[b + 1] - cu[b]
        for h in range(H):
            at = np.arange(L) if keep is None else np.nonzero(keep[h, cu[b]:cu[b + 1]].cpu().numpy())[0]
            at = at[:cap]
            pg, off = slots_of(st, b, len(at), page)
            t = torch.from_numpy(at + cu[b]).long()
            for pool, src, sc in (("k_pages", k, "k_scale"), ("v_pages", v, "v_scale")):
                rows = src[t, h]
                if st[pool].dtype == E4M3:
                    st[pool].view(torch.uint8)[pg, h, off] = quantise(rows, E4M3, float(st[sc][h]) if st.get(sc) is not None else 1.0).view(torch.uint8)
                else:
                    st[pool][pg, h, off] = rows
            st["pos"][pg, h, off] = torch.from_numpy(at).to(torch.int32)
            if st.get("weight") is not None:
                st["weight"][pg, h, off] = 0.0 if score is None else score.cpu()[h, t]
            st["count"][b, h] = len(at)
            st["seen"][b, h] = L
    return st


def assert_same_state(a, st, what=""):
    for name in ("k_pages", "v_pages", "pos", "weight", "count", "seen"):
        if a.get(name) is None:
            continue
        x, y = as_bytes(a[name]), as_bytes(st[name])
        assert np.array_equal(x, y), f"{what}: {name} differs in {int((x != y).sum())} of {x.size} values"
