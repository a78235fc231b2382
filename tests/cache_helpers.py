"""Inputs and the 64-bit oracle of the key/value cache tests (plain loops over sequences and heads,
nothing shared with the kernels)."""
from __future__ import annotations

import math

import torch

D = 128
HALF_BF16 = 2.0 ** -8   # a rounding to bf16 is off by at most this much of the value
HALF_FP32 = 2.0 ** -24


def make(lens, new, hq, hkv, page, seed, fill=float("nan"), extra_pages=2, max_pages=None, scale=1.0, k_gain=1.0,
         device="cpu"):
    """A cache of several sequences in randomly ordered pages. Slots that no sequence uses hold `fill`
    (NaN by default: nothing may read them into a result), in K, V, weights and positions (-77)."""
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    tot = [a + b for a, b in zip(lens, new)]
    need = [-(-t // page) for t in tot]
    num_pages = sum(need) + extra_pages
    width = max_pages or max(1, max(need))
    perm = torch.randperm(num_pages, generator=g)
    table = torch.full((S, width), -5, dtype=torch.int32)
    k = torch.full((num_pages * page, hkv, D), fill, dtype=torch.bfloat16)
    v = torch.full((num_pages * page, hkv, D), fill, dtype=torch.bfloat16)
    w = torch.full((num_pages, hkv, page), fill, dtype=torch.float32)
    pos = torch.full((num_pages, hkv, page), -77, dtype=torch.int32)
    at = 0
    for s in range(S):
        table[s, :need[s]] = perm[at:at + need[s]].to(torch.int32)
        at += need[s]
        r = rows(table, page, s, tot[s])
        k[r] = (torch.randn((tot[s], hkv, D), generator=g) * k_gain).to(torch.bfloat16)
        v[r] = torch.randn((tot[s], hkv, D), generator=g).to(torch.bfloat16)
        w[r // page, :, r % page] = torch.rand((tot[s], hkv), generator=g)
        pos[r // page, :, r % page] = torch.arange(tot[s], dtype=torch.int32)[:, None].expand(-1, hkv)
    T = sum(new)
    q = (torch.randn((T, hq, D), generator=g) * scale).to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"lens": list(lens), "new": list(new), "hq": hq, "hkv": hkv, "page": page, "table": table, "k": k, "v": v,
            "w": w, "pos": pos, "q": q, "cu": cu, "num_pages": num_pages}


def rows(table, page, s, n):
    u = torch.arange(n)
    return table[s].long()[u // page] * page + u % page


def oracle_attn(x, scale=None, decay=None):
    """out, lse, weights in 64 bits, and bounds of the kernel's error for each, from the number formats:
    out: the tensor cores take P in bf16 (HALF_BF16 of every term p |v|) and the result is rounded once
    more (HALF_BF16 |o|); scores are sums of 128 products in fp32 (128 roundings of at most HALF_FP32 of
    the sum of |q_i k_i|), scaled (2 roundings), exponentiated by a unit good to 2^-22."""
    hq, hkv, page = x["hq"], x["hkv"], x["page"]
    G, scale = hq // hkv, scale or 1 / math.sqrt(D)
    T = sum(x["new"])
    out = torch.zeros((T, hq, D), dtype=torch.float64)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64)
    w = x["w"].double().clone()
    b_out, b_lse, b_w = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(w)
    for s, (c, L) in enumerate(zip(x["lens"], x["new"])):
        if L == 0:
            continue
        n = c + L
        r = rows(x["table"], page, s, n)
        t0 = x["cu"][s]
        for g in range(hkv):
            k, v = x["k"][r, g].double(), x["v"][r, g].double()
            add, err = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
            for h in range(g * G, (g + 1) * G):
                q = x["q"][t0:t0 + L, h].double()
                sc = (q @ k.T) * scale
                mag = (q.abs() @ k.abs().T) * scale
                ok = torch.arange(n)[None, :] <= (c + torch.arange(L))[:, None]
                sc = sc.masked_fill(~ok, -math.inf)
                z = torch.logsumexp(sc, 1)
                p = torch.exp(sc - z[:, None])
                # relative error of one term: its score (and the row's reference, as large) and the exponential
                ds = torch.where(ok, mag * (130 * HALF_FP32) + sc.abs().nan_to_num(posinf=0.0) * 4 * HALF_FP32,
                                 torch.zeros_like(mag)).amax(1)
                rel = 2 * ds + 8 * HALF_FP32
                out[t0:t0 + L, h] = p @ v
                pv = p @ v.abs()
                b_out[t0:t0 + L, h] = (out[t0:t0 + L, h].abs() * HALF_BF16 + pv * HALF_BF16 * (1 + HALF_BF16)
                                       + pv * (2 * rel[:, None] + n * HALF_FP32)) * 1.01
                lse[h, t0:t0 + L] = z
                b_lse[h, t0:t0 + L] = rel + (n + 8) * HALF_FP32 + 4 * HALF_FP32 * z.abs()
                add += p.sum(0)
                tot = rel + b_lse[h, t0:t0 + L] + (L * G + 8) * HALF_FP32
                err += (p * tot[:, None]).sum(0)
            if decay is not None:
                old = w[r // page, g, r % page]
                w[r // page, g, r % page] = add if decay == 0 else old * decay + add
                b_w[r // page, g, r % page] = err + (4 * HALF_FP32) * (add + (0 if decay == 0 else old.abs()))
    return out, lse, w, b_out, b_lse, b_w


def oracle_select(x, budget, sinks, recent, next_pos):
    """moves, counts, new lens by a plain sort in Python."""
    S, hkv, page = len(x["lens"]), x["hkv"], x["page"]
    moves = torch.full((S, hkv, budget, 2), -1, dtype=torch.int32)
    counts = torch.zeros((S, hkv), dtype=torch.int32)
    lens = torch.zeros(S, dtype=torch.int32)
    for s, (c, L) in enumerate(zip(x["lens"], x["new"])):
        n = c + L
        lens[s] = min(n, budget)
        if n <= budget:
            continue
        r = rows(x["table"], page, s, n)
        end = next_pos[s] + L
        for g in range(hkv):
            w = x["w"][r // page, g, r % page].tolist()
            pos = x["pos"][r // page, g, r % page].tolist()

            def key(u):
                safe = pos[u] < sinks or pos[u] >= end - recent
                val = w[u]
                nan = val != val
                return (0 if safe else 1, 1 if (nan and not safe) else 0, 0.0 if (safe or nan) else -val, u)
            kept = sorted(sorted(range(n), key=key)[:budget])
            stay = [u for u in kept if u >= budget]
            below = set(kept)
            gone = [u for u in range(budget) if u not in below]
            counts[s, g] = len(stay)
            for i, (a, b) in enumerate(zip(stay, gone)):
                moves[s, g, i, 0], moves[s, g, i, 1] = a, b
    return moves, counts, lens


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
