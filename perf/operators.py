"""Cases of the key/value cache operators: attention of new tokens over a paged cache (with the
attention weight that each cached token collects), append, selection by that weight, compaction.

A case names one call: its heads, page size and sequence lengths. The lengths of a ragged batch come
from case["shape"] (a number that seeds them), so that the work is known without the inputs.
"""
import math
import random

import torch

own = False

D = 128  # head dimension of the framework


# ----------------------------------------------------------------------------- shapes of a case
def _ragged(rng, lo, hi, n):
    """n lengths in [lo, hi], spread over their logarithm."""
    return [min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))
            for _ in range(n)]


def _shapes(case):
    """Per sequence: tokens cached before the call and new tokens."""
    rng = random.Random(case["shape"])
    cached = _ragged(rng, case["len_lo"] + 1, case["len_hi"] + 1, case["seqs"])
    new = _ragged(rng, case["new_lo"] + 1, case["new_hi"] + 1, case["seqs"])
    return [c - 1 for c in cached], [n - 1 for n in new]


def listed():
    base = {"hq": 32, "hkv": 8, "page": 64, "shape": 1}
    return [
        # one user's chat: a single new token over a short context, where latency is all that counts
        {**base, "name": "attn_token_2k", "op": "attn", "seqs": 1, "len_lo": 2047, "len_hi": 2047, "new_lo": 1,
         "new_hi": 1, "weights": False},
        # the ordinary serving step: one new token each for a batch of requests of very different lengths
        {**base, "name": "attn_tokens_batch", "op": "attn", "seqs": 32, "len_lo": 500, "len_hi": 16000, "new_lo": 1,
         "new_hi": 1, "weights": False, "shape": 2},
        # one long document: a single token over 128K keys, collecting the weight that eviction ranks by
        {**base, "name": "attn_token_128k_weights", "op": "attn", "seqs": 1, "len_lo": 131071, "len_hi": 131071,
         "new_lo": 1, "new_hi": 1, "weights": True, "page": 128},
        # mixed batch (single tokens, drafts to verify, prompt pieces), small pages, six heads over two
        {**base, "name": "attn_mixed_ragged", "op": "attn", "seqs": 13, "len_lo": 0, "len_hi": 9000, "new_lo": 1,
         "new_hi": 700, "weights": False, "hq": 6, "hkv": 2, "page": 16, "shape": 5},
        # a prompt piece over a long cached prefix that is no multiple of any block
        {**base, "name": "attn_chunk_4096", "op": "attn", "seqs": 1, "len_lo": 28611, "len_hi": 28611, "new_lo": 4096,
         "new_hi": 4096, "weights": False, "page": 256},
        # the last tokens of a prompt as observers: the weight that each prompt token gets from them
        {**base, "name": "attn_window_weights", "op": "attn", "seqs": 2, "len_lo": 20000, "len_hi": 32700,
         "new_lo": 64, "new_hi": 64, "weights": True, "shape": 3},
        # one new token of each request of a batch goes into the cache
        {**base, "name": "append_tokens", "op": "append", "seqs": 64, "len_lo": 100, "len_hi": 2000, "new_lo": 1,
         "new_hi": 1, "weights": True},
        # whole prompts of ragged lengths go into the cache
        {**base, "name": "append_prompts", "op": "append", "seqs": 6, "len_lo": 0, "len_hi": 300, "new_lo": 1000,
         "new_hi": 16000, "weights": True, "shape": 4},
        # caches a little over their budget after some decode steps
        {**base, "name": "select_decode", "op": "select", "seqs": 16, "len_lo": 4100, "len_hi": 4200, "new_lo": 1,
         "new_hi": 1, "weights": True, "budget": 4096, "sinks": 4, "recent": 1024},
        # a long prompt is cut down to the budget it decodes with
        {**base, "name": "select_128k", "op": "select", "seqs": 1, "len_lo": 131071, "len_hi": 131071, "new_lo": 1,
         "new_hi": 1, "weights": True, "budget": 16384, "sinks": 4, "recent": 2000, "page": 128},
        # the same two, applied to the keys, values, weights and positions
        {**base, "name": "compact_decode", "op": "compact", "seqs": 16, "len_lo": 4100, "len_hi": 4200, "new_lo": 1,
         "new_hi": 1, "weights": True, "budget": 4096, "sinks": 4, "recent": 1024},
        {**base, "name": "compact_128k", "op": "compact", "seqs": 1, "len_lo": 131071, "len_hi": 131071, "new_lo": 1,
         "new_hi": 1, "weights": True, "budget": 16384, "sinks": 4, "recent": 2000, "page": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "select", "compact"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (6, 2), (4, 1), (8, 8), (16, 2), (40, 8)])
    case = {"op": op, "hq": hq, "hkv": hkv, "page": rng.choice([16, 32, 48, 64, 128, 192, 256]),
            "shape": rng.randrange(1 << 30), "weights": True}
    if op == "attn":
        case["weights"] = rng.random() < 0.5
        kind = rng.choice(["tokens", "drafts", "chunks"])
        case["seqs"] = _log(rng, 1, 48 if kind == "tokens" else 12)
        new = 1 if kind == "tokens" else _log(rng, 2, 12) if kind == "drafts" else _log(rng, 13, 2000)
        case["new_hi"] = new
        case["new_lo"] = rng.choice([new, max(1, new // 5), 0 if new > 1 else 1])
        top = _log(rng, 40, 120000 // case["seqs"])
        if kind == "chunks":  # no more pairs than the largest listed case
            top = min(top, int(1.2e8 / (case["seqs"] * new * (hq / 32))) + 40)
        case["len_hi"] = top
        case["len_lo"] = rng.choice([0, top // 7, top])
    elif op == "append":
        case["seqs"] = _log(rng, 1, 64)
        case["new_hi"] = _log(rng, 1, 30000 // case["seqs"])
        case["new_lo"] = rng.choice([0 if case["new_hi"] > 1 else 1, case["new_hi"]])
        case["len_hi"] = _log(rng, 1, 2000)
        case["len_lo"] = 0
    else:
        case["seqs"] = _log(rng, 1, 24)
        top = _log(rng, 60, 130000 // case["seqs"])
        case["len_hi"] = top
        case["len_lo"] = rng.choice([top, top // 2])
        case["new_lo"], case["new_hi"] = rng.choice([(0, 0), (1, 1), (1, 30)])
        case["budget"] = max(20, int(top * rng.uniform(0.1, 1.05)))
        case["sinks"] = rng.randrange(0, 9)
        case["recent"] = rng.randrange(0, case["budget"] // 2)
    if case["op"] in ("attn", "append") and sum(_shapes(case)[1]) == 0:  # every sequence drew no new token
        case["new_lo"] = case["new_hi"]
    return case


# ----------------------------------------------------------------------------- inputs
def _starts(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    hq, hkv, page, S = case["hq"], case["hkv"], case["page"], case["seqs"]
    cached, new = _shapes(case)
    total = [c + n for c, n in zip(cached, new)]
    T = sum(new)
    need = [max(1, -(-t // page)) for t in total]
    num_pages, max_pages = sum(need) + 2, max(need)
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((S, max_pages), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n

    def normal(*shape, scale=1.0):
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        return x if scale == 1.0 else x * scale

    st = {"case": case, "cached": cached, "new": new, "table": table}
    rows = num_pages * page
    if case["op"] == "select":  # ranks weights and positions only: the smallest cache that can carry them
        st["k_cache"] = st["v_cache"] = torch.zeros((rows, hkv, D), dtype=torch.bfloat16, device=dev)
    else:
        st["k_cache"], st["v_cache"] = normal(rows, hkv, D), normal(rows, hkv, D)
    st["lens"] = torch.tensor(cached, dtype=torch.int32, device=dev)
    st["next_pos"] = st["lens"].clone()
    st["weights"] = st["positions"] = None
    if case["weights"]:
        # collected softmax weight has a heavy tail, and tokens that nothing attends share tiny values
        w = torch.exp(2.0 * torch.randn((num_pages, hkv, page), generator=gen, device=dev) - 4.0)
        st["weights"] = torch.where(w < 2e-3, torch.round(w * 2048.0) / 2048.0, w)
        st["positions"] = torch.zeros((num_pages, hkv, page), dtype=torch.int32, device=dev)
    if case["op"] == "attn":
        st["q"] = normal(max(T, 1), hq, D)[:T]
        # keys that a query leans on, as in a trained model: some rows of the cache are much larger
        heavy = torch.rand((rows, 1, 1), generator=gen, device=dev) < 0.02
        st["k_cache"] = torch.where(heavy, st["k_cache"] * 2.5, st["k_cache"]).contiguous()
        st["out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros((hq, T), dtype=torch.float32, device=dev)
    elif case["op"] == "append":
        st["k"], st["v"] = normal(max(T, 1), hkv, D)[:T], normal(max(T, 1), hkv, D)[:T]
    else:
        # tokens were evicted before: every head holds its own positions, rising but with gaps, in an
        # order that earlier compactions have shuffled
        for s in range(S):
            n = total[s]
            st["next_pos"][s] = n + n // 3 - new[s]
            pos = torch.stack([torch.randperm(n + n // 3, generator=gen, device=dev)[:n] for _ in range(hkv)])
            _write_slots(st["positions"], table[s], page, n, pos.to(torch.int32))
        B = case["budget"]
        st["moves"] = torch.full((S, hkv, B, 2), -1, dtype=torch.int32, device=dev)
        st["move_counts"] = torch.zeros((S, hkv), dtype=torch.int32, device=dev)
        st["new_lens"] = torch.zeros(S, dtype=torch.int32, device=dev)
        if case["op"] == "compact":
            _plain_select(st)
    if own:
        import block_sparse_long_causal_b200 as fp
        p = fp.problem(_starts(new), hq, hkv, D, 128)
        c = fp.kv_cache(p, st["k_cache"], st["v_cache"], st["lens"], table, page, weights=st["weights"],
                        positions=st["positions"])
        st["p"], st["c"] = p, c
        if case["op"] == "attn":
            st["workspace"] = torch.empty(fp.cache_attn_workspace(p, c), dtype=torch.uint8, device=dev)
    return st


# ----------------------------------------------------------------------------- the plain form
def _slots(x, pages, page, n):
    """[num_pages, heads, page] -> [heads, n] in slot order of one sequence."""
    g = x[pages[:-(-n // page)].long()] if n else x[:0]
    return g.permute(1, 0, 2).reshape(x.shape[1], -1)[:, :n]


def _write_slots(x, pages, page, n, val):
    if n == 0:
        return
    u = torch.arange(n, device=x.device)
    x[pages.long()[u // page], :, u % page] = val.T.to(x.dtype)


def _rows(pages, page, u):
    return pages.long()[u // page] * page + u % page


def _plain_attn(st):
    case = st["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    G, scale = hq // hkv, 1.0 / math.sqrt(D)
    t0 = 0
    for s, (c, L) in enumerate(zip(st["cached"], st["new"])):
        if L == 0:
            continue
        n, dev = c + L, st["q"].device
        rows = _rows(st["table"][s], page, torch.arange(n, device=dev))
        acc = torch.zeros((hkv, n), device=dev)
        # heads one at a time, queries in pieces: the scores of a long chunk fill the card otherwise
        for g in range(hkv):
            k = st["k_cache"][rows, g].float()
            v = st["v_cache"][rows, g].float()
            step = max(1, (1 << 28) // (n * G))
            for a in range(0, L, step):
                b = min(L, a + step)
                q = st["q"][t0 + a:t0 + b, g * G:(g + 1) * G].float().reshape(-1, D)
                sc = (q @ k.T) * scale
                if L > 1:
                    late = torch.arange(n, device=dev)[None, :] > (c + torch.arange(a, b, device=dev))[:, None]
                    sc = sc.view(b - a, G, n).masked_fill_(late[:, None, :], -math.inf).view(-1, n)
                m = sc.amax(dim=1, keepdim=True)
                e = torch.exp(sc - m)
                l = e.sum(dim=1, keepdim=True)
                st["out"][t0 + a:t0 + b, g * G:(g + 1) * G] = ((e @ v) / l).view(b - a, G, D).to(torch.bfloat16)
                st["lse"][g * G:(g + 1) * G, t0 + a:t0 + b] = (m + torch.log(l)).view(b - a, G).T
                if case["weights"]:
                    acc[g] += (e / l).sum(dim=0)
        if case["weights"]:
            _write_slots(st["weights"], st["table"][s], page, n, acc)
        t0 += L


def _plain_append(st):
    page, t0 = st["case"]["page"], 0
    for s, (c, L) in enumerate(zip(st["cached"], st["new"])):
        if L:
            u = torch.arange(c, c + L, device=st["k"].device)
            rows = _rows(st["table"][s], page, u)
            st["k_cache"][rows] = st["k"][t0:t0 + L]
            st["v_cache"][rows] = st["v"][t0:t0 + L]
            pg = st["table"][s].long()[u // page]
            st["weights"][pg, :, u % page] = 0.0
            pos = st["next_pos"][s] + torch.arange(L, device=u.device, dtype=torch.int32)
            st["positions"][pg, :, u % page] = pos[:, None]
        t0 += L


def _plain_select(st):
    case = st["case"]
    B, page, hkv = case["budget"], case["page"], case["hkv"]
    st["moves"].fill_(-1)
    for s, (c, L) in enumerate(zip(st["cached"], st["new"])):
        n = c + L
        st["new_lens"][s] = min(n, B)
        st["move_counts"][s] = 0
        if n <= B:
            continue
        w = _slots(st["weights"], st["table"][s], page, n)
        pos = _slots(st["positions"], st["table"][s], page, n)
        safe = (pos < case["sinks"]) | (pos >= st["next_pos"][s] + L - case["recent"])
        rank = torch.where(safe, math.inf, w)
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :B]
        keep = torch.zeros((hkv, n), dtype=torch.bool, device=w.device).scatter_(1, order, True)
        for g in range(hkv):
            src = torch.nonzero(keep[g, B:]).flatten() + B
            dst = torch.nonzero(~keep[g, :B]).flatten()
            st["moves"][s, g, :len(src), 0] = src.to(torch.int32)
            st["moves"][s, g, :len(src), 1] = dst.to(torch.int32)
            st["move_counts"][s, g] = len(src)


def _plain_compact(st):
    page = st["case"]["page"]
    for s in range(st["case"]["seqs"]):
        pages = st["table"][s].long()
        for g in range(st["case"]["hkv"]):
            mv = st["moves"][s, g]
            mv = mv[mv[:, 0] >= 0].long()
            src, dst = mv[:, 0], mv[:, 1]
            for x in (st["k_cache"], st["v_cache"]):
                x[_rows(pages, page, dst), g] = x[_rows(pages, page, src), g]
            for x in (st["weights"], st["positions"]):
                x[pages[dst // page], g, dst % page] = x[pages[src // page], g, src % page]
    st["lens"].copy_(st["new_lens"])


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import block_sparse_long_causal_b200 as fp
        p, c = st["p"], st["c"]
        if op == "attn":
            # decay 0: the weights of this call alone, so that a pass gives the same however often it runs
            fp.cache_attn(p, c, st["q"], 0.0, st["workspace"], st["out"], st["lse"],
                          decay=0.0 if case["weights"] else None)
        elif op == "append":
            fp.cache_append(p, c, st["k"], st["v"], st["next_pos"])
        elif op == "select":
            fp.cache_select(p, c, case["budget"], case["sinks"], case["recent"], st["next_pos"], st["moves"],
                            st["move_counts"], st["new_lens"])
        else:
            fp.cache_compact(p, c, case["budget"], st["moves"], st["move_counts"], st["new_lens"])
    else:
        {"attn": _plain_attn, "append": _plain_append, "select": _plain_select, "compact": _plain_compact}[op](st)
    return _outputs(st)


def _outputs(st):
    op = st["case"]["op"]
    if op == "attn":
        return (st["out"], st["lse"], st["weights"]) if st["case"]["weights"] else (st["out"], st["lse"])
    if op == "append":
        return st["k_cache"], st["v_cache"], st["weights"], st["positions"]
    if op == "select":
        return st["moves"], st["move_counts"], st["new_lens"]
    return st["k_cache"], st["v_cache"], st["weights"], st["positions"], st["lens"]


# ----------------------------------------------------------------------------- work
def work(case):
    hq, hkv = case["hq"], case["hkv"]
    cached, new = _shapes(case)
    total = [c + n for c, n in zip(cached, new)]
    T = sum(new)
    if case["op"] == "attn":
        keys = sum(t for t, n in zip(total, new) if n)
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
        b = keys * hkv * D * 4 + T * hq * (D * 4 + 4)
        if case["weights"]:
            b += keys * hkv * 4
        return {"bytes": b, "flops": 4 * D * hq * pairs}
    if case["op"] == "append":
        return {"bytes": T * hkv * (D * 8 + 8), "flops": 0}
    B = case["budget"]
    over = [(t, t - B) for t in total if t > B]
    # slots past the budget that stay: the recent ones and the heaviest, spread evenly over the slots
    moved = sum(e * B // t for t, e in over) * hkv
    if case["op"] == "select":
        return {"bytes": sum(t for t, _ in over) * hkv * 8 + case["seqs"] * hkv * (B * 8 + 4), "flops": 0}
    return {"bytes": moved * (2 * (D * 4 + 8) + 8) + 4 * case["seqs"], "flops": 0}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    table, page, hkv = st["table"].cpu().tolist(), case["page"], case["hkv"]

    def row(s, u):
        return table[s][u // page] * page + u % page

    if case["op"] == "attn":
        G = case["hq"] // hkv
        q, kc, vc = st["q"].double(), st["k_cache"], st["v_cache"]
        out, lse = torch.zeros_like(st["out"], dtype=torch.float64), torch.zeros_like(st["lse"], dtype=torch.float64)
        wts = st["weights"].double() if case["weights"] else None
        first = 0
        for s in range(case["seqs"]):
            n, L = st["cached"][s] + st["new"][s], st["new"][s]
            if L == 0:
                continue
            idx = torch.tensor([row(s, u) for u in range(n)], device=q.device)
            for h in range(case["hq"]):
                k, v = kc[idx, h // G].double(), vc[idx, h // G].double()
                if wts is not None and h % G == 0:
                    wts[idx // page, h // G, idx % page] = 0.0
                piece = max(1, (1 << 26) // n)
                for a in range(0, L, piece):
                    b = min(L, a + piece)
                    x = torch.einsum("td,ud->tu", q[first + a:first + b, h], k) / D ** 0.5
                    seen = torch.arange(n, device=q.device) <= torch.arange(n - L + a, n - L + b, device=q.device)[:, None]
                    x = torch.where(seen, x, -torch.inf)
                    z = torch.logsumexp(x, dim=1)
                    p = torch.exp(x - z[:, None])
                    lse[h, first + a:first + b] = z
                    out[first + a:first + b, h] = p @ v
                    if wts is not None:
                        wts[idx // page, h // G, idx % page] += p.sum(dim=0)
            first += L
        return (out, lse, wts) if case["weights"] else (out, lse)
    if case["op"] == "append":
        k, v = st["k_cache"].double(), st["v_cache"].double()
        w, pos = st["weights"].double(), st["positions"].clone()
        at, slots = [], []
        for s in range(case["seqs"]):
            for t in range(st["new"][s]):
                at.append(row(s, st["cached"][s] + t))
                slots.append(st["cached"][s] + t)
        at = torch.tensor(at, device=k.device, dtype=torch.long)
        k[at], v[at] = st["k"].double(), st["v"].double()
        w[at // page, :, at % page] = 0.0
        pos[at // page, :, at % page] = torch.tensor(slots, device=k.device, dtype=torch.int32)[:, None].expand(-1, hkv)
        return k, v, w, pos
    if case["op"] == "select":
        B = case["budget"]
        moves, counts = torch.full_like(st["moves"], -1).cpu(), torch.zeros_like(st["move_counts"]).cpu()
        lens = torch.zeros_like(st["new_lens"]).cpu()
        weights, positions = st["weights"].cpu().double(), st["positions"].cpu()
        for s in range(case["seqs"]):
            n = st["cached"][s] + st["new"][s]
            lens[s] = min(n, B)
            if n <= B:
                continue
            idx = torch.tensor([row(s, u) for u in range(n)])
            end = int(st["next_pos"][s]) + st["new"][s]
            for g in range(hkv):
                w, pos = weights[idx // page, g, idx % page].tolist(), positions[idx // page, g, idx % page].tolist()
                rank = sorted(range(n), key=lambda u: (
                    not (pos[u] < case["sinks"] or pos[u] >= end - case["recent"]), -w[u], u))
                kept = sorted(rank[:B])
                gone = sorted(set(range(B)) - set(kept))
                stay = [u for u in kept if u >= B]
                counts[s, g] = len(stay)
                if stay:
                    moves[s, g, :len(stay)] = torch.tensor(list(zip(stay, gone)), dtype=torch.int32)
        dev = st["moves"].device
        return moves.to(dev), counts.to(dev), lens.to(dev)
    k, v = st["k_cache"].double(), st["v_cache"].double()
    w, pos = st["weights"].double(), st["positions"].clone()
    counts, moves = st["move_counts"].cpu().tolist(), st["moves"].cpu().tolist()
    for s in range(case["seqs"]):
        for g in range(hkv):
            mv = moves[s][g][:counts[s][g]]
            if not mv:
                continue
            a = torch.tensor([row(s, m[0]) for m in mv], device=k.device)
            b = torch.tensor([row(s, m[1]) for m in mv], device=k.device)
            k[b, g], v[b, g] = k[a, g], v[a, g]
            w[b // page, g, b % page] = w[a // page, g, a % page]
            pos[b // page, g, b % page] = pos[a // page, g, a % page]
    return k, v, w, pos, st["new_lens"].clone()
