"""Key/value cache operators on the GPU against the plain 64-bit oracle of cache_helpers.py. Unused
slots, pages and table entries hold NaN or out-of-range values throughout."""
import math

import pytest
import torch

import block_sparse_long_causal_b200 as fp
from cache_helpers import D, bits, make, oracle_attn, oracle_select, rows

pytestmark = pytest.mark.gpu


class Dev:
    """A case of cache_helpers.make on the GPU."""

    def __init__(self, x, weights=True, positions=True, max_len=0):
        self.x = x
        self.k, self.v = x["k"].cuda(), x["v"].cuda()
        self.w = x["w"].cuda() if weights else None
        self.pos = x["pos"].cuda() if positions else None
        self.lens = torch.tensor(x["lens"], dtype=torch.int32, device="cuda")
        self.table = x["table"].cuda()
        self.p = fp.problem(x["cu"], x["hq"], x["hkv"])
        self.c = fp.kv_cache(self.p, self.k, self.v, self.lens, self.table, x["page"], self.w, self.pos, max_len)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((max(1, fp.cache_attn_workspace(self.p, self.c)),), 0xFF, dtype=torch.uint8, device="cuda")

    def attn(self, q=None, decay=None, scale=0.0, lse=True):
        T = self.p.total_tokens
        out = torch.full((T, self.x["hq"], D), 7.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((self.x["hq"], T), 7.0, device="cuda") if lse else None
        fp.cache_attn(self.p, self.c, self.x["q"].cuda() if q is None else q, scale, self.ws, out, ls, decay, self.st)
        return out, ls

    def status(self):
        torch.cuda.synchronize()
        return int(self.st.item())


def check_attn(x, out, lse, w=None, decay=None, scale=None):
    o, z, ww, bo, bz, bw = oracle_attn(x, scale, decay)
    eo = (out.cpu().double() - o).abs()
    assert bool((eo <= bo).all()), f"out: {(eo - bo).max().item()} over its bound"
    if lse is not None:
        ez = (lse.cpu().double() - z).abs()
        assert bool((ez <= bz).all()), f"lse: {(ez - bz).max().item()} over its bound"
    if w is not None:
        used = bw > 0
        ew = (w.cpu().double() - ww).abs()
        assert bool((ew[used] <= bw[used]).all()), f"weights: {(ew[used] - bw[used]).max().item()} over their bound"
        assert torch.equal(bits(w.cpu())[~used], bits(x["w"])[~used]), "weights of other slots changed"


# lens, new, hq, hkv, page
ATTN = [
    ([0], [1], 4, 2, 16),                                   # a first token
    ([1], [1], 4, 2, 16),
    ([15, 16, 17], [1, 1, 1], 4, 2, 16),                    # around a page's end
    ([63, 64, 65, 127, 128, 129], [1] * 6, 8, 2, 48),       # around the tiles' ends
    ([2047], [1], 32, 8, 64),
    ([700, 0, 33, 1500], [1, 0, 1, 1], 6, 2, 32),           # a sequence without new tokens
    ([300, 9], [3, 4], 8, 2, 16),                           # exactly 12 and 16 rows
    ([300, 9], [5, 2], 8, 2, 64),                           # past 16 rows
    ([0, 5], [37, 200], 4, 1, 16),                          # whole prompts
    ([130, 1000, 40], [129, 33, 1], 32, 8, 64),
    ([257], [300], 6, 2, 192),                              # three heads a group
    ([900, 20], [40, 1], 40, 8, 256),                       # five heads a group
    ([77], [90], 8, 8, 16),                                 # one head a group
    ([100, 3], [2, 70], 64, 1, 128),                        # 64 heads a group
    ([511], [513], 16, 2, 128),
    ([3000, 17, 512, 0, 90, 700, 5, 260], [200, 150, 1, 300, 64, 90, 33, 170], 32, 8, 48),  # more units than CTAs
    ([6000], [20], 2, 2, 16),                               # one row tile, two warpgroups, split over many CTAs
    ([128, 384, 383], [32, 128, 1], 4, 1, 64),              # keys and rows that fill their tiles exactly
    ([1000, 64, 0], [8, 1, 5], 8, 2, 16),                   # exactly 32 rows
    ([63, 640], [31, 17], 2, 2, 48),                        # 31 rows, one head a group
    ([4000, 5], [11, 2], 6, 2, 16),                         # one row more than 32
]


@pytest.mark.parametrize("lens,new,hq,hkv,page", ATTN)
def test_attention_matches_the_oracle(lens, new, hq, hkv, page):
    x = make(lens, new, hq, hkv, page, seed=len(lens) + lens[0])
    d = Dev(x)
    out, lse = d.attn()
    assert d.status() == 0
    check_attn(x, out, lse)
    assert torch.equal(bits(d.w.cpu()), bits(x["w"]))  # decay None leaves the weights alone


@pytest.mark.parametrize("decay", [0.0, 0.75, 1.0])
@pytest.mark.parametrize("lens,new,hq,hkv,page", ATTN[2:])
def test_collected_weights_match_the_oracle(lens, new, hq, hkv, page, decay):
    x = make(lens, new, hq, hkv, page, seed=3 + lens[0])
    if decay == 0.0:  # the old weight is not read
        x["w"].fill_(float("nan"))
    d = Dev(x)
    out, lse = d.attn(decay=decay, lse=False)
    assert d.status() == 0
    check_attn(x, out, lse, d.w, decay)


def test_scale_and_large_scores():
    # near one-hot rows: the maximum grows late and by much, so that the rescaling path runs
    x = make([800, 100], [1, 60], 8, 2, 32, seed=9, k_gain=6.0)
    d = Dev(x)
    out, lse = d.attn(decay=1.0, scale=0.21)
    assert d.status() == 0
    check_attn(x, out, lse, d.w, 1.0, 0.21)


def test_rows_of_a_fused_projection_and_max_len():
    x = make([90, 10], [5, 70], 8, 2, 16, seed=12, max_pages=9)
    fused = torch.full((75, 8 + 2 + 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :8] = x["q"].cuda()
    d = Dev(x, max_len=95)
    out, lse = d.attn(q=fused[:, :8], decay=0.0)
    assert d.status() == 0
    check_attn(x, out, lse, d.w, 0.0)


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 90, (1024,), generator=g).tolist()
    new = torch.randint(0, 3, (1024,), generator=g).tolist()
    new[5] = 40
    x = make(lens, new, 4, 2, 16, seed=4)
    d = Dev(x)
    out, lse = d.attn(decay=1.0)
    assert d.status() == 0
    check_attn(x, out, lse, d.w, 1.0)


def test_same_bits_on_every_run_and_on_another_stream():
    x = make([5000, 700, 0], [1, 90, 17], 32, 8, 64, seed=2)
    d = Dev(x)
    a, la = d.attn(decay=0.0)
    wa = d.w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, lb = d.attn(decay=0.0)
    torch.cuda.current_stream().wait_stream(side)
    assert d.status() == 0
    assert torch.equal(bits(a), bits(b)) and torch.equal(bits(la), bits(lb)) and torch.equal(bits(wa), bits(d.w))


def test_captured_step_replays_as_the_sequences_grow():
    """One captured append + attention, replayed with lens advanced on the device."""
    lens, steps = [30, 61], 5
    x = make(lens, [steps, steps], 8, 2, 16, seed=21)
    full_k, full_v, q = x["k"].clone(), x["v"].clone(), x["q"]
    for s in range(2):  # the new slots are empty until they are appended
        r = rows(x["table"], 16, s, lens[s] + steps)[lens[s]:]
        x["k"][r] = float("nan")
        x["v"][r] = float("nan")
    k, v, w, pos = x["k"].cuda(), x["v"].cuda(), x["w"].cuda(), x["pos"].cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nxt = torch.tensor([40, 99], dtype=torch.int32, device="cuda")
    p = fp.problem([0, 1, 2], 8, 2)
    c = fp.kv_cache(p, k, v, ln, x["table"].cuda(), 16, w, pos)
    ws = torch.empty(fp.cache_attn_workspace(p, c), dtype=torch.uint8, device="cuda")
    qs = torch.empty((2, 8, D), dtype=torch.bfloat16, device="cuda")
    ks, vs = (torch.empty((2, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty_like(qs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        fp.cache_append(p, c, ks, vs, nxt, st)
        fp.cache_attn(p, c, qs, 0.0, ws, out, None, 1.0, st)
        ln.add_(1)
        nxt.add_(1)

    for t in (qs, ks, vs):
        t.zero_()
    keep = [t.clone() for t in (k, v, w, pos, ln, nxt)]
    step()  # warm-up outside the capture, undone below
    torch.cuda.synchronize()
    for a, b in zip((k, v, w, pos, ln, nxt), keep):
        a.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for s in range(2):
            r = rows(x["table"], 16, s, lens[s] + i + 1)[-1]
            qs[s].copy_(q[s * steps + i])
            ks[s].copy_(full_k[r])
            vs[s].copy_(full_v[r])
        graph.replay()
        torch.cuda.synchronize()
        y = dict(x, k=full_k, v=full_v, lens=[a + i for a in lens], new=[1, 1], cu=[0, 1, 2],
                 q=torch.stack([q[i], q[steps + i]]))
        check_attn(y, out, None)
        assert ln.tolist() == [a + i + 1 for a in lens]
    assert int(st.item()) == 0
    for s in range(2):
        r = rows(x["table"], 16, s, lens[s] + steps)[lens[s]:]
        assert pos.cpu()[r // 16, :, r % 16].tolist() == [[[40, 99][s] + i] * 2 for i in range(steps)]


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements whose sequence sits in its last pages."""
    hkv, page, n = 8, 256, 700
    pages = (1 << 31) // (hkv * D * page) + 8
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.zeros((pages * page, hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    x = {"lens": [n], "new": [4], "hq": 8, "hkv": hkv, "page": page, "cu": [0, 4], "table": table.cpu()}
    r = rows(x["table"], page, 0, n + 4).cuda()
    kk = torch.randn((n + 4, hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    vv = torch.randn((n + 4, hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    k[r[:n]], v[r[:n]] = kk[:n], vv[:n]
    w = torch.zeros((pages, hkv, page), device="cuda")
    pos = torch.zeros((pages, hkv, page), dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    p = fp.problem(x["cu"], 8, hkv)
    c = fp.kv_cache(p, k, v, lens, table, page, w, pos)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp.cache_append(p, c, kk[n:], vv[n:], None, st)
    q = torch.randn((4, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(fp.cache_attn_workspace(p, c), dtype=torch.uint8, device="cuda")
    fp.cache_attn(p, c, q, 0.0, ws, out, None, 0.0, st)
    B = 300
    mv = torch.empty((1, hkv, B, 2), dtype=torch.int32, device="cuda")
    cnt, nl = torch.empty((1, hkv), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    fp.cache_select(p, c, B, 2, 20, None, mv, cnt, nl, st)
    x.update(q=q.cpu(), k=None, v=None, w=None)
    small = dict(x, table=torch.tensor([[0, 1, 2]], dtype=torch.int32), k=torch.zeros((3 * page, hkv, D), dtype=torch.bfloat16),
                 v=torch.zeros((3 * page, hkv, D), dtype=torch.bfloat16), w=torch.zeros((3, hkv, page)),
                 pos=torch.zeros((3, hkv, page), dtype=torch.int32))
    small["k"][:n + 4], small["v"][:n + 4] = kk.cpu(), vv.cpu()
    check_attn(small, out, None)
    idx = table[0].long()
    small["w"], small["pos"] = w[idx].cpu(), pos[idx].cpu()
    # only the appended slots have positions: the others hold 0, which counts as a sink
    m2, c2, l2 = oracle_select(small, B, 2, 20, [n])
    assert torch.equal(mv.cpu(), m2) and torch.equal(cnt.cpu(), c2) and torch.equal(nl.cpu(), l2)
    fp.cache_compact(p, c, B, mv, cnt, nl, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and lens.tolist() == [B]
    rr = rows(x["table"], page, 0, n + 4)
    for h in range(hkv):
        want = kk[:, h].clone()
        pairs = m2[0, h, :int(c2[0, h])].long()
        want[pairs[:, 1].cuda()] = want[pairs[:, 0].cuda()]
        assert torch.equal(bits(k[rr.cuda(), h]), bits(want))
    del k, v, w, pos
    torch.cuda.empty_cache()


@pytest.mark.parametrize("lens,new,hq,hkv", [([40], [4], 8, 2), ([200], [12], 2, 2), ([90], [7], 8, 2),
                                             ([70, 33], [200, 60], 8, 2), ([300], [20], 4, 2)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_masked_values_reach_nobody(lens, new, hq, hkv, value):
    """A non-finite V of a new token is seen by the rows from that token on, and by no row before it."""
    x = make(lens, new, hq, hkv, 16, seed=23)
    G = hq // hkv
    clean, clean_lse = Dev(x).attn()
    s, j, g, cols = 0, new[0] // 2, hkv - 1, [0, 5, 63, 64, 127]
    y = dict(x, v=x["v"].clone())
    r = int(rows(x["table"], 16, s, lens[s] + j + 1)[-1])
    y["v"][r, g, cols] = value
    d = Dev(y)
    out, lse = d.attn()
    assert d.status() == 0 and torch.equal(bits(lse.cpu()), bits(clean_lse.cpu()))
    want = clean.clone()
    for c in cols:
        want[j:new[0], g * G:(g + 1) * G, c] = value
    got, want = out.cpu(), want.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(bits(got.nan_to_num(nan=1.0)), bits(want.nan_to_num(nan=1.0)))
    # and a K of it: NaN rows from the token on, the others within their bounds
    y = dict(x, k=x["k"].clone())
    y["k"][r, g, 3] = math.nan
    d = Dev(y)
    out, lse = d.attn()
    bad = torch.zeros(out.shape[:2], dtype=torch.bool)
    bad[j:new[0], g * G:(g + 1) * G] = True
    assert torch.equal(out.cpu().isnan().all(-1), bad) and torch.equal(lse.cpu().isnan(), bad.T)
    o, z, _, bo, bz, _ = oracle_attn(x)
    assert bool(((out.cpu().double() - o).abs() <= bo)[~bad].all())
    assert bool(((lse.cpu().double() - z).abs() <= bz)[~bad.T].all())


def test_noted_values_stay_with_their_unit():
    """A CTA takes several units one after another, the last of them often in part and without the slots of its new
    tokens: what an earlier unit noted of its non-finite V must not reach it."""
    S, hq, hkv = 512, 8, 2
    g = torch.Generator().manual_seed(41)
    lens, new = torch.randint(100, 900, (S,), generator=g).tolist(), torch.randint(9, 21, (S,), generator=g).tolist()
    x = make(lens, new, hq, hkv, 16, seed=42)
    o, _, _, bound, _, _ = oracle_attn(x)
    y = dict(x, v=x["v"].clone())
    odd = torch.zeros(o.shape, dtype=torch.float64)  # what a row gets by itself
    for s in range(S):
        j, h, col = s % new[s], s % hkv, (37 * s) % D
        value = (math.nan, math.inf, -math.inf)[s % 3]
        y["v"][int(rows(x["table"], 16, s, lens[s] + j + 1)[-1]), h, col] = value
        t0 = x["cu"][s]
        odd[t0 + j:t0 + new[s], h * 4:(h + 1) * 4, col] = value
    want = o + odd
    d = Dev(y)
    for _ in range(3):
        out, _ = d.attn()
        assert d.status() == 0
        got = out.cpu().double()
        fin = want.isfinite()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got[~fin].nan_to_num(nan=1.0), want[~fin].nan_to_num(nan=1.0))
        assert bool(((got - o).abs() <= bound)[fin].all())


# short drafts (few rows), longer pieces (row tiles, several of them), heads that fill a tile and that do not
ODD_ROWS = [([40], [4], 8, 2), ([200, 17], [12, 1], 2, 2), ([130], [20], 4, 2), ([300], [90], 6, 2), ([70, 33], [200, 60], 8, 2)]


@pytest.mark.parametrize("lens,new,hq,hkv", ODD_ROWS)
def test_a_query_that_is_nan_reaches_the_weights_of_the_slots_it_sees(lens, new, hq, hkv):
    x = make(lens, new, hq, hkv, 16, seed=29)
    _, _, w, _, _, bound = oracle_attn(x, None, 0.5)
    j, h = new[0] // 3, hq - 1
    y = dict(x, q=x["q"].clone())
    y["q"][j, h, 7] = math.nan
    d = Dev(y)
    _, lse = d.attn(decay=0.5)
    assert d.status() == 0
    nan_lse = torch.zeros(lse.shape, dtype=torch.bool)
    nan_lse[h, j] = True
    assert torch.equal(lse.cpu().isnan(), nan_lse)
    seen = torch.zeros(w.shape, dtype=torch.bool)
    r = rows(x["table"], 16, 0, lens[0] + j + 1)
    seen[r // 16, hkv - 1, r % 16] = True
    got, used = d.w.cpu().double(), bound > 0
    assert torch.equal(got.isnan() & used, seen)
    assert bool(((got - w).abs() <= bound)[used & ~seen].all())


@pytest.mark.parametrize("lens,new,hq,hkv", ODD_ROWS)
def test_a_row_without_a_finite_score_adds_no_weight(lens, new, hq, hkv):
    """All scores of one row are -inf: its sum is 0, its lse -inf, and it leaves the slots' weights alone."""
    x = make(lens, new, hq, hkv, 16, seed=30)
    j, h = new[0] // 3, hq - 1
    x["k"][:, hkv - 1, 0] = x["k"][:, hkv - 1, 0].abs() + 0.25
    x["q"][j, h] = 0.0
    _, _, w, _, _, bound = oracle_attn(x, None, 0.5)
    r = rows(x["table"], 16, 0, lens[0] + j + 1)
    w[r // 16, hkv - 1, r % 16] -= 1.0 / (lens[0] + j + 1)  # the row of zeros gave every slot the same
    y = dict(x, q=x["q"].clone())
    y["q"][j, h, 0] = -math.inf
    d = Dev(y)
    out, lse = d.attn(decay=0.5)
    assert d.status() == 0
    assert float(lse[h, j]) == -math.inf and not bool(out[j, h].any())
    got, used = d.w.cpu().double(), bound > 0
    assert bool(((got - w).abs() <= bound)[used].all())


@pytest.mark.parametrize("lens,new,hq,hkv", [([40], [4], 8, 2), ([200], [70], 8, 2), ([300], [90], 6, 2), ([257], [130], 10, 2),
                                             ([900], [6], 22, 2)])
def test_an_infinite_key_that_every_row_scores_at_minus_infinity(lens, new, hq, hkv):
    """Its slot is left with its decayed weight, also where the heads of a group do not fill a row tile."""
    x = make(lens, new, hq, hkv, 16, seed=33)
    G, u = hq // hkv, lens[0] // 2
    x["q"][:, :G, 5] = x["q"][:, :G, 5].abs() + 1
    r = int(rows(x["table"], 16, 0, u + 1)[-1])
    # for the oracle a score so low that its exponential is nothing, in place of -inf
    x["k"][r, 0, 5] = -1024.0
    o, z, w, bo, bz, bw = oracle_attn(x, None, 0.5)
    assert float(w[r // 16, 0, r % 16] - 0.5 * x["w"][r // 16, 0, r % 16].double()) < 2.0 ** -100
    y = dict(x, k=x["k"].clone())
    y["k"][r, 0, 5] = -math.inf
    d = Dev(y)
    out, lse = d.attn(decay=0.5)
    assert d.status() == 0
    assert bool(((out.cpu().double() - o).abs() <= bo).all()) and bool(((lse.cpu().double() - z).abs() <= bz).all())
    used = bw > 0
    assert bool(((d.w.cpu().double() - w).abs() <= bw)[used].all())


def test_prompt_pieces_capture_and_replay():
    """A captured append + attention + selection + compaction of prompt pieces, replayed on other inputs."""
    lens, new, hq, hkv, page, B = [30, 261], [70, 50], 8, 2, 16, 200
    x = make(lens, new, hq, hkv, page, seed=5)
    d = Dev(x)
    T = sum(new)
    mv = torch.empty((2, hkv, B, 2), dtype=torch.int32, device="cuda")
    cnt, nl = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((2, hkv), (2,)))
    q, out = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((T, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        fp.cache_append(d.p, d.c, k, v, None, d.st)
        fp.cache_attn(d.p, d.c, q, 0.0, d.ws, out, None, 0.0, d.st)
        fp.cache_select(d.p, d.c, B, 2, 60, None, mv, cnt, nl, d.st)
        fp.cache_compact(d.p, d.c, B, mv, cnt, nl, d.st)

    keep = [t.clone() for t in (d.k, d.v, d.w, d.pos, d.lens)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        for t, src in zip((d.k, d.v, d.w, d.pos, d.lens), keep):
            t.copy_(src)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        y = dict(x, q=q.cpu(), k=x["k"].clone(), v=x["v"].clone(), w=x["w"].clone())
        t0 = 0
        for s in range(2):
            r = rows(x["table"], page, s, lens[s] + new[s])[lens[s]:]
            y["k"][r], y["v"][r] = k.cpu()[t0:t0 + new[s]], v.cpu()[t0:t0 + new[s]]
            t0 += new[s]
        graph.replay()
        assert d.status() == 0
        check_attn(y, out, None)
        assert d.lens.tolist() == [100, 200]
        assert cnt[0].tolist() == [0] * hkv and min(cnt[1].tolist()) >= 50  # of 60 recent ones past slot 200


def test_calls_of_two_streams_at_once():
    """Two callers, each with its own workspace, on streams of their own."""
    xs = [make([900, 40], [1, 1], 8, 2, 16, seed=1), make([500, 77], [90, 30], 8, 2, 32, seed=2)]
    ds = [Dev(x) for x in xs]
    qs = [x["q"].cuda() for x in xs]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, q, o, st in zip(ds, qs, outs, streams):
            fp.cache_attn(d.p, d.c, q, 0.0, d.ws, o, None, 0.0, d.st, stream=st)
    for x, d, o in zip(xs, ds, outs):
        assert d.status() == 0
        check_attn(x, o, None, d.w, 0.0)


def test_wait_that_runs_out_is_flagged_and_the_context_survives(monkeypatch):
    x = make([300], [70], 8, 2, 16, seed=3)
    d = Dev(x)
    good, _ = d.attn(decay=0.0)
    assert d.status() == 0
    monkeypatch.setenv("FP_TEST_UNSIGNALLED_WAIT", "1")
    monkeypatch.setenv("FP_WAIT_LIMIT_MS", "50")
    d.attn(decay=0.0)
    assert d.status() & fp.FP_DEV_TIMEOUT
    monkeypatch.delenv("FP_TEST_UNSIGNALLED_WAIT")
    monkeypatch.delenv("FP_WAIT_LIMIT_MS")
    d.st.zero_()
    again, _ = d.attn(decay=0.0)
    assert d.status() == 0 and torch.equal(bits(good), bits(again))


def test_bad_tables_are_flagged_and_leave_the_outputs():
    x = make([100, 40], [1, 1], 4, 2, 16, seed=6)
    d = Dev(x, max_len=101)
    d.lens[0] = 101  # with the new token one more than max_len
    out, lse = d.attn(decay=1.0)
    assert d.status() & fp.FP_DEV_BAD_PROBLEM
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all()) and torch.equal(bits(d.w.cpu()), bits(x["w"]))
    # a page outside the cache reads as zeros: the other sequence is as it was
    d = Dev(x)
    d.table[0, 2] = x["num_pages"]
    out, lse = d.attn()
    assert d.status() & fp.FP_DEV_BAD_PROBLEM
    y = dict(x, table=x["table"].clone(), k=torch.cat([x["k"], torch.zeros((16, 2, D), dtype=torch.bfloat16)]),
             v=torch.cat([x["v"], torch.zeros((16, 2, D), dtype=torch.bfloat16)]),
             w=torch.cat([x["w"], torch.zeros((1, 2, 16))]))
    y["table"][0, 2] = x["num_pages"]
    check_attn(y, out, lse)


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("lens,new,hq,hkv,page", [ATTN[0], ATTN[2], ATTN[5], ATTN[8], ATTN[11], ATTN[13]])
@pytest.mark.parametrize("arrays", [True, False])
def test_append_writes_its_slots_and_nothing_else(lens, new, hq, hkv, page, arrays):
    x = make(lens, new, hq, hkv, page, seed=8)
    d = Dev(x, weights=arrays, positions=arrays)
    T, g = sum(new), torch.Generator().manual_seed(1)
    fused = torch.randn((T, hq + 2 * hkv, D), generator=g).to(torch.bfloat16)
    nxt = torch.arange(len(lens), dtype=torch.int32) * 1000
    fc = fused.cuda()
    fp.cache_append(d.p, d.c, fc[:, hq:hq + hkv], fc[:, hq + hkv:], nxt.cuda(), d.st)
    assert d.status() == 0
    k, v, w, pos = x["k"].clone(), x["v"].clone(), x["w"].clone(), x["pos"].clone()
    t = 0
    for s in range(len(lens)):
        for i in range(new[s]):
            u = lens[s] + i
            pg = int(x["table"][s, u // page])
            k[pg * page + u % page], v[pg * page + u % page] = fused[t, hq:hq + hkv], fused[t, hq + hkv:]
            w[pg, :, u % page], pos[pg, :, u % page] = 0.0, int(nxt[s]) + i
            t += 1
    assert torch.equal(bits(d.k.cpu()), bits(k)) and torch.equal(bits(d.v.cpu()), bits(v))
    if arrays:
        assert torch.equal(bits(d.w.cpu()), bits(w)) and torch.equal(d.pos.cpu(), pos)


def test_append_skips_and_flags_what_has_no_slot():
    x = make([20, 40], [2, 1], 4, 2, 16, seed=8)
    d = Dev(x)
    d.table[0, 1] = -1  # the page of both new tokens of sequence 0
    kv = torch.ones((3, 2, D), dtype=torch.bfloat16, device="cuda")
    fp.cache_append(d.p, d.c, kv, kv, None, d.st)
    assert d.status() & fp.FP_DEV_BAD_PROBLEM
    changed = (bits(d.k.cpu()) != bits(x["k"])).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(rows(x["table"], 16, 1, 41)[-1])]


# ----------------------------------------------------------------------------- selection, compaction
def select_case(seed, lens, new, hkv, page, kind):
    x = make(lens, new, hkv, hkv, page, seed=seed)
    g = torch.Generator().manual_seed(seed)
    w = x["w"]
    if kind == "ties":
        w.copy_(torch.where(w.isnan(), w, (w * 4).floor() / 4))
    elif kind == "equal":
        w.fill_(0.5)
    elif kind == "odd":  # signs, zeros of both signs, infinities, NaN, the smallest and largest numbers
        vals = torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, 3.4e38, -3.4e38])
        w.copy_(vals[torch.randint(0, len(vals), w.shape, generator=g)])
    elif kind == "tail":
        w.copy_(torch.exp(3 * torch.randn(w.shape, generator=g)))
    nxt = []
    for s, (c, L) in enumerate(zip(lens, new)):  # positions in any order, with gaps
        n = c + L
        r = rows(x["table"], page, s, n)
        for h in range(hkv):
            x["pos"][r // page, h, r % page] = torch.randperm(n + n // 2 + 1, generator=g)[:n].to(torch.int32)
        nxt.append(n + n // 2 + 1 - L)
    return x, nxt


SELECT = [
    # lens, new, hkv, page, budget, sinks, recent
    ([40], [1], 2, 16, 40, 0, 0),           # one over
    ([39, 40, 3], [1, 1, 0], 2, 16, 40, 2, 5),
    ([0, 1, 2], [0, 0, 1], 1, 16, 1, 0, 0),
    ([0, 1, 2], [0, 0, 1], 1, 16, 1, 0, 1),
    ([500, 900], [0, 7], 3, 48, 130, 4, 126),  # nothing but protected slots stays
    ([3000], [1], 2, 64, 700, 4, 100),
    ([3000, 2000, 50], [30, 0, 1], 2, 32, 1999, 0, 0),
    ([9000], [0], 1, 128, 33, 1, 3),
    ([70000, 12], [3, 1], 2, 32, 9001, 4, 500),  # several CTAs a head
]


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "tail"])
@pytest.mark.parametrize("lens,new,hkv,page,budget,sinks,recent", SELECT)
def test_selection_and_compaction(lens, new, hkv, page, budget, sinks, recent, kind):
    x, nxt = select_case(17 + budget, lens, new, hkv, page, kind)
    d = Dev(x)
    S = len(lens)
    moves = torch.full((S, hkv, budget, 2), 99, dtype=torch.int32, device="cuda")
    cnt = torch.full((S, hkv), 99, dtype=torch.int32, device="cuda")
    nl = torch.full((S,), 99, dtype=torch.int32, device="cuda")
    nd = torch.tensor(nxt, dtype=torch.int32, device="cuda")
    fp.cache_select(d.p, d.c, budget, sinks, recent, nd, moves, cnt, nl, d.st)
    assert d.status() == 0
    m, c, ln = oracle_select(x, budget, sinks, recent, nxt)
    assert torch.equal(cnt.cpu(), c) and torch.equal(nl.cpu(), ln) and torch.equal(moves.cpu(), m)
    for t, name in ((d.k, "k"), (d.v, "v"), (d.w, "w")):
        assert torch.equal(bits(t.cpu()), bits(x[name]))  # nothing of the cache changed yet
    fp.cache_compact(d.p, d.c, budget, moves, cnt, nl, d.st)
    assert d.status() == 0 and d.lens.tolist() == ln.tolist()
    k, v, w, pos = x["k"].clone(), x["v"].clone(), x["w"].clone(), x["pos"].clone()
    for s in range(S):
        for h in range(hkv):
            for a, b in m[s, h, :int(c[s, h])].tolist():
                pa, pb = (int(x["table"][s, u // page]) for u in (a, b))
                k[pb * page + b % page, h], v[pb * page + b % page, h] = (
                    t[pa * page + a % page, h] for t in (x["k"], x["v"]))
                w[pb, h, b % page], pos[pb, h, b % page] = x["w"][pa, h, a % page], x["pos"][pa, h, a % page]
    assert torch.equal(bits(d.k.cpu()), bits(k)) and torch.equal(bits(d.v.cpu()), bits(v))
    assert torch.equal(bits(d.w.cpu()), bits(w)) and torch.equal(d.pos.cpu(), pos)


@pytest.mark.parametrize("kind", ["ties", "tail"])
def test_selection_of_more_slots_than_shared_memory_holds(kind):
    """Many heads of a long sequence: one CTA a head, which reads its slots again in every pass."""
    n, hkv, page, B, sinks, recent = 30001, 160, 256, 4000, 4, 900
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(9)
    w = torch.rand((pages, hkv, page), generator=g, device="cuda")
    w = (w * 50).floor() / 50 if kind == "ties" else torch.exp(8 * w)
    pos = torch.stack([torch.randperm(pages * page, generator=g, device="cuda") for _ in range(hkv)]).to(torch.int32)
    pos = pos.view(hkv, pages, page).transpose(0, 1).contiguous()
    k = torch.zeros((pages * page, hkv, D), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    lens, nxt = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (n, pages * page))
    p = fp.problem([0, 0], hkv, hkv)
    c = fp.kv_cache(p, k, k, lens, table, page, w, pos)
    mv = torch.empty((1, hkv, B, 2), dtype=torch.int32, device="cuda")
    cnt, nl = torch.empty((1, hkv), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp.cache_select(p, c, B, sinks, recent, nxt, mv, cnt, nl, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and nl.tolist() == [B]
    for h in (0, 77, 159):
        x = {"lens": [n], "new": [0], "hkv": 1, "page": page, "table": table.cpu(), "w": w[:, h:h + 1].cpu(),
             "pos": pos[:, h:h + 1].cpu()}
        m, cc, _ = oracle_select(x, B, sinks, recent, [pages * page])
        assert torch.equal(mv[:, h:h + 1].cpu(), m) and int(cnt[0, h]) == int(cc)


@pytest.mark.parametrize("kind", ["ties", "tail"])
@pytest.mark.parametrize("S,hkv,n,width,B", [
    (1, 8, 300000, 0, 4000),       # a cluster a head, a large part of the keys in every CTA
    (1, 3, 200001, 0, 150000),
    (1, 8, 800001, 0, 20000),      # clusters that read their slots again in every pass
    (16, 8, 3000, 131072, 1000),   # short sequences with a block table for long ones
    (16, 8, 40001, 131072, 5000),
    (20, 8, 30000, 0, 3000),       # more heads than the GPU holds at once
    (1, 160, 60001, 0, 4000),      # the same, read again in every pass
])
def test_selection_by_what_the_gpu_holds(S, hkv, n, width, B, kind):
    page, sinks, recent = 256, 4, B // 3
    need = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(n + B)
    table = torch.full((S, max(need, width // page)), -9, dtype=torch.int32, device="cuda")
    table[:, :need] = torch.randperm(S * need, generator=g, device="cuda").view(S, need).to(torch.int32)
    w = torch.rand((S * need, hkv, page), generator=g, device="cuda")
    w = (w * 50).floor() / 50 if kind == "ties" else torch.exp(8 * w)
    pos = torch.randint(0, 2 * n, w.shape, generator=g, dtype=torch.int32, device="cuda")
    k = torch.empty((S * need * page, hkv, D), dtype=torch.bfloat16, device="cuda")  # selection does not read it
    lens, nxt = (torch.full((S,), v, dtype=torch.int32, device="cuda") for v in (n, 2 * n))
    p = fp.problem([0] * (S + 1), hkv, hkv)
    c = fp.kv_cache(p, k, k, lens, table, page, w, pos)
    mv = torch.empty((S, hkv, B, 2), dtype=torch.int32, device="cuda")
    cnt, nl = torch.empty((S, hkv), dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp.cache_select(p, c, B, sinks, recent, nxt, mv, cnt, nl, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and nl.tolist() == [B] * S
    for s, h in {(0, 0), (S - 1, hkv - 1), (S // 2, hkv // 3)}:
        x = {"lens": [n], "new": [0], "hkv": 1, "page": page, "table": table[s:s + 1].cpu(), "w": w[:, h:h + 1].cpu(),
             "pos": pos[:, h:h + 1].cpu()}
        m, cc, _ = oracle_select(x, B, sinks, recent, [2 * n])
        assert int(cnt[s, h]) == int(cc) and torch.equal(mv[s, h].cpu(), m[0, 0])


def test_selection_without_positions_ranks_slots():
    x, _ = select_case(5, [300], [1], 2, 16, "plain")
    d = Dev(x, positions=False)
    n = 301
    r = rows(x["table"], 16, 0, n)
    x["pos"][r // 16, :, r % 16] = torch.arange(n, dtype=torch.int32)[:, None].expand(-1, 2)
    mv = torch.empty((1, 2, 64, 2), dtype=torch.int32, device="cuda")
    cnt, nl = torch.empty((1, 2), dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    fp.cache_select(d.p, d.c, 64, 4, 16, None, mv, cnt, nl, d.st)
    m, c, ln = oracle_select(x, 64, 4, 16, [300])
    assert d.status() == 0 and torch.equal(mv.cpu(), m) and torch.equal(cnt.cpu(), c) and torch.equal(nl.cpu(), ln)


def test_compaction_skips_and_flags_bad_moves():
    x, _ = select_case(5, [60], [0], 1, 16, "plain")
    d = Dev(x)
    mv = torch.full((1, 1, 16, 2), -1, dtype=torch.int32, device="cuda")
    # a source below the budget, a source past the cache, destinations out of range; one good move
    for i, (a, b) in enumerate([(3, 2), (1 << 30, 1), (20, -1), (20, 16), (-9, 0), (40, 5)]):
        mv[0, 0, i, 0], mv[0, 0, i, 1] = a, b
    cnt = torch.tensor([[6]], dtype=torch.int32, device="cuda")
    fp.cache_compact(d.p, d.c, 16, mv, cnt, torch.tensor([16], dtype=torch.int32, device="cuda"), d.st)
    assert d.status() & fp.FP_DEV_BAD_LIST
    r = rows(x["table"], 16, 0, 60)
    k = x["k"].clone()
    k[r[5]] = x["k"][r[40]]
    assert torch.equal(bits(d.k.cpu()), bits(k)) and d.lens.tolist() == [16]
    cnt[0, 0] = 1 << 30  # a count past the list: flagged, nothing read past the list
    mv.fill_(-1)
    d.st.zero_()
    fp.cache_compact(d.p, d.c, 16, mv, cnt, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"), d.st)
    assert d.status() & fp.FP_DEV_BAD_LIST and d.status() & fp.FP_DEV_BAD_PROBLEM
    assert torch.equal(bits(d.k.cpu()), bits(k)) and d.lens.tolist() == [16]


# ----------------------------------------------------------------------------- a run of them together
def test_prompt_then_budgeted_decode():
    """A prompt through the block-sparse chunked prefill, the weight that its last tokens give, the cache
    cut to a budget, then decode steps that append, attend, collect and evict, next to a plain model of
    the same cache in 64 bits."""
    hq, hkv, page, L, budget, sinks, recent, steps = 8, 2, 128, 700, 256, 4, 32, 12
    x = make([0], [L], hq, hkv, page, seed=31, fill=0.0, max_pages=8)
    prompt = Dev(x)
    pc = fp.paged_cache(prompt.p, [0], x["table"].clamp(min=0).numpy(), page, x["num_pages"])
    nb = prompt.p.total_blocks
    qp = torch.empty((nb, hq, D), device="cuda")
    kp = torch.empty((pc.total_kv_blocks, hkv, D), device="cuda")
    cnts = torch.zeros((hq, nb), dtype=torch.int32, device="cuda")
    idx = torch.zeros(pc.index_elems, dtype=torch.int32, device="cuda")
    out = torch.empty((L, hq, D), dtype=torch.bfloat16, device="cuda")
    q = x["q"].cuda()
    fp.paged_block_pool(prompt.p, pc, q, prompt.k, qp, kp)
    fp.paged_block_search(prompt.p, pc, qp, kp, 0.2, cnts, idx, prompt.st)
    fp.paged_block_sparse_attn(prompt.p, pc, q, prompt.k, prompt.v, cnts, idx, 0.0, out, None, prompt.st)
    assert prompt.status() == 0 and bool(out.isfinite().all())
    # the last 16 tokens observe the whole prompt
    obs = dict(x, lens=[L - 16], new=[16], cu=[0, 16], q=x["q"][-16:])
    d = Dev(obs)
    o, lse = d.attn(decay=0.0)
    assert d.status() == 0
    check_attn(obs, o, lse, d.w, 0.0)
    # eviction to the budget, against the oracle on the weights that the GPU collected
    y = dict(obs, w=d.w.cpu(), pos=d.pos.cpu(), k=d.k.cpu(), v=d.v.cpu())
    mv = torch.empty((1, hkv, budget, 2), dtype=torch.int32, device="cuda")
    cnt, nl = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((1, hkv), (1,)))
    nxt = torch.tensor([L - 16], dtype=torch.int32, device="cuda")
    ln = d.lens
    one = fp.problem([0, 1], hq, hkv)
    c1 = fp.kv_cache(one, d.k, d.v, ln, d.table, page, d.w, d.pos)
    ws = torch.empty(fp.cache_attn_workspace(one, c1), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(77)

    def evict(p, c, state):
        fp.cache_select(p, c, budget, sinks, recent, nxt, mv, cnt, nl, d.st)
        want = oracle_select(state, budget, sinks, recent, nxt.tolist())
        assert torch.equal(mv.cpu(), want[0]) and torch.equal(cnt.cpu(), want[1])
        fp.cache_compact(p, c, budget, mv, cnt, nl, d.st)
        assert ln.tolist() == want[2].tolist()

    evict(d.p, d.c, y)
    nxt += 16
    for i in range(steps):
        new = [torch.randn((1, n, D), generator=g).to(torch.bfloat16) for n in (hq, hkv, hkv)]
        fp.cache_append(one, c1, new[1].cuda(), new[2].cuda(), nxt, d.st)
        o = torch.empty((1, hq, D), dtype=torch.bfloat16, device="cuda")
        z = torch.empty((hq, 1), device="cuda")
        before = d.w.cpu()
        fp.cache_attn(one, c1, new[0].cuda(), 0.0, ws, o, z, 1.0, d.st)
        state = dict(x, lens=ln.tolist(), new=[1], cu=[0, 1], q=new[0], k=d.k.cpu(), v=d.v.cpu(), w=before)
        check_attn(state, o, z, d.w, 1.0)
        state.update(w=d.w.cpu(), pos=d.pos.cpu())
        evict(one, c1, state)
        nxt += 1
        r = rows(x["table"], page, 0, budget)
        held = d.pos.cpu()[r // page, :, r % page]
        for h in range(hkv):  # sinks and the latest tokens are there, and nothing twice
            have = held[:, h].tolist()
            assert len(set(have)) == budget and set(range(sinks)) <= set(have)
            assert set(range(L + i + 1 - recent, L + i + 1)) <= set(have)
    assert d.status() == 0


@pytest.mark.parametrize("hq,hkv,page,B,L", [(8, 2, 16, 64, 1), (6, 2, 48, 200, 9), (4, 4, 64, 200, 40)])
def test_chained_steps_equal_steps_that_wait(hq, hkv, page, B, L):
    """Kernels of consecutive calls overlap at their ends: the same steps with a synchronisation after every
    call leave the same bits."""
    S, steps = 2, 20
    need = -(-(B + L) // page)
    g = torch.Generator().manual_seed(B + L)
    table = torch.randperm(S * need, generator=g).view(S, need).to(torch.int32).cuda()
    k, v = (torch.randn((S * need * page, hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.rand((S * need, hkv, page), generator=g).cuda()
    pos = torch.arange(need * page, dtype=torch.int32).view(1, need, 1, page).expand(S, need, hkv, page)
    inv = torch.empty_like(table.flatten().long())
    inv[table.flatten().long()] = torch.arange(S * need, device="cuda")
    pos = pos.reshape(S * need, hkv, page).cuda()[inv].contiguous()
    lens = torch.tensor([B - 5, B // 2], dtype=torch.int32, device="cuda")
    nxt = lens.clone()
    p = fp.problem([0, L, 2 * L], hq, hkv)
    c = fp.kv_cache(p, k, v, lens, table, page, w, pos)
    ws = torch.empty(fp.cache_attn_workspace(p, c), dtype=torch.uint8, device="cuda")
    mv = torch.empty((S, hkv, B, 2), dtype=torch.int32, device="cuda")
    cnt, nl = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((S, hkv), (S,)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qs, ks, vs = (torch.randn((steps, S * L, n, D), generator=g).to(torch.bfloat16).cuda() for n in (hq, hkv, hkv))
    state = (k, v, w, pos, lens, nxt)
    start = [t.clone() for t in state]

    def run(wait):
        for t, a in zip(state, start):
            t.copy_(a)
        outs = torch.empty_like(qs)
        for i in range(steps):
            for call in (lambda: fp.cache_append(p, c, ks[i], vs[i], nxt, st),
                         lambda: fp.cache_attn(p, c, qs[i], 0.0, ws, outs[i], None, 0.9, st),
                         lambda: fp.cache_select(p, c, B, 2, B // 4, nxt, mv, cnt, nl, st),
                         lambda: fp.cache_compact(p, c, B, mv, cnt, nl, st), lambda: nxt.add_(L)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [bits(outs)] + [bits(t).clone() for t in state]

    want = run(True)
    assert int(st.item()) == 0 and lens.tolist() == [B, min(B, B // 2 + steps * L)]
    for _ in range(2):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


def test_chained_evictions_equal_evictions_that_wait():
    """Append, selection and compaction one after another without an attention between them: a selection reads
    the weights and positions that the compaction before it has just moved, the next append the lengths."""
    S, hkv, page, n0, steps = 4, 8, 16, 4000, 24
    need = n0 // page + 2
    g = torch.Generator().manual_seed(51)
    table = torch.randperm(S * need, generator=g).view(S, need).to(torch.int32).cuda()
    k, v = (torch.randn((S * need * page, hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.rand((S * need, hkv, page), generator=g).cuda()
    pos = torch.randint(0, n0, w.shape, generator=g, dtype=torch.int32).cuda()
    lens = torch.tensor([n0, n0 - 1, n0 - 700, 1500], dtype=torch.int32, device="cuda")
    nxt = torch.full((S,), n0, dtype=torch.int32, device="cuda")
    p = fp.problem(list(range(S + 1)), hkv, hkv)
    c = fp.kv_cache(p, k, v, lens, table, page, w, pos)
    budgets = [n0 - 150 * i for i in range(1, steps + 1)]
    bufs = [(torch.empty((S, hkv, B, 2), dtype=torch.int32, device="cuda"),
             torch.empty((S, hkv), dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda"))
            for B in budgets]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ks, vs = (torch.randn((steps, S, hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    state = (k, v, w, pos, lens)
    start = [t.clone() for t in state]

    def run(wait):
        for t, a in zip(state, start):
            t.copy_(a)
        for i, (B, b) in enumerate(zip(budgets, bufs)):
            for call in (lambda: fp.cache_append(p, c, ks[i], vs[i], nxt, st),
                         lambda: fp.cache_select(p, c, B, 4, 40, nxt, *b, st), lambda: fp.cache_compact(p, c, B, *b, st)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [bits(t).clone() for t in state] + [t.clone() for b in bufs for t in b]

    want = run(True)
    assert int(st.item()) == 0 and lens.tolist() == [budgets[-1]] * S and min(int(b[1].min()) for b in bufs[-8:]) > 0
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
