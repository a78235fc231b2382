"""Key/value cache calls: what they refuse on the host, before any launch (no GPU needed)."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_sparse_long_causal_b200 as fp

OK, NULL = C.c_void_p(4096), None


def _err():
    return fp._lib.fp_last_error().decode()


def _problem(cu=(0, 3, 3, 10), hq=8, hkv=2):
    p = fp.fp_problem()
    host = np.array(cu, np.int32)
    assert fp._lib.fp_problem_init(C.byref(p), host.ctypes.data_as(C.c_void_p), len(cu) - 1, C.c_void_p(16), hq, hkv,
                                   128, 128) == fp.FP_OK
    return p, host


def _cache(cu=(0, 3, 3, 10), max_pages=8, page_size=48, num_pages=16, max_len=0, k=OK, v=OK, lens=OK, table=OK,
           host=None):
    p, h = _problem(cu)
    h = h if host is None else np.array(host, np.int32)
    c = fp.fp_kv_cache()
    st = fp._lib.fp_kv_cache_init(C.byref(c), C.byref(p), h.ctypes.data_as(C.c_void_p), k, v, lens, table, max_pages,
                                  page_size, num_pages, max_len)
    return st, p, c


def test_init_fills_the_description():
    st, p, c = _cache()
    assert st == fp.FP_OK, _err()
    assert (c.max_pages, c.page_size, c.num_pages, c.max_len, c.max_new) == (8, 48, 16, 8 * 48, 7)
    assert not c.weights and not c.positions
    st, _, c = _cache(max_len=100)
    assert st == fp.FP_OK and c.max_len == 100


@pytest.mark.parametrize("kw,status", [
    (dict(k=NULL), fp.FP_ERR_INVALID_ARG), (dict(v=NULL), fp.FP_ERR_INVALID_ARG),
    (dict(lens=NULL), fp.FP_ERR_INVALID_ARG), (dict(table=NULL), fp.FP_ERR_INVALID_ARG),
    (dict(k=C.c_void_p(4104)), fp.FP_ERR_INVALID_ARG),
    (dict(page_size=0), fp.FP_ERR_UNSUPPORTED), (dict(page_size=8), fp.FP_ERR_UNSUPPORTED),
    (dict(page_size=40), fp.FP_ERR_UNSUPPORTED), (dict(page_size=-16), fp.FP_ERR_UNSUPPORTED),
    (dict(max_pages=0), fp.FP_ERR_INVALID_ARG), (dict(num_pages=0), fp.FP_ERR_INVALID_ARG),
    (dict(num_pages=1 << 26), fp.FP_ERR_INVALID_ARG),
    (dict(max_len=-1), fp.FP_ERR_INVALID_ARG), (dict(max_len=8 * 48 + 1), fp.FP_ERR_INVALID_ARG),
    (dict(max_len=6), fp.FP_ERR_INVALID_ARG),                # a sequence brings 7 new tokens
    (dict(host=(0, 3, 3, 9)), fp.FP_ERR_INVALID_ARG), (dict(host=(0, 4, 3, 10)), fp.FP_ERR_INVALID_ARG),
])
def test_init_refuses(kw, status):
    st, _, _ = _cache(**kw)
    assert st == status and _err()


def test_calls_refuse_bad_arguments_before_launch():
    st, p, c = _cache()
    assert st == fp.FP_OK
    P, K, L = C.byref(p), C.byref(c), fp._lib
    bad = fp.FP_ERR_INVALID_ARG
    mis = C.c_void_p(4098)
    n = C.c_int64(0)
    assert L.fp_cache_attn_workspace(P, K, C.byref(n)) == fp.FP_OK and n.value > 0
    assert L.fp_cache_attn_workspace(P, K, None) == bad and L.fp_cache_attn_workspace(P, None, C.byref(n)) == bad
    f = C.c_float

    def attn(q=OK, qs=0, scale=0.0, ws=OK, wb=None, out=OK, lse=NULL, decay=-1.0, cache=K):
        return L.fp_cache_attn(P, cache, q, qs, f(scale), ws, n.value if wb is None else wb, out, lse, f(decay), NULL,
                               NULL)
    assert attn(cache=None) == bad and attn(q=NULL) == bad and attn(out=NULL) == bad
    assert attn(q=mis) == bad and attn(out=mis) == bad
    assert attn(qs=8 * 128 - 8) == bad and attn(qs=8 * 128 + 4) == bad and attn(qs=-1024) == bad
    assert attn(scale=float("nan")) == bad and attn(scale=float("inf")) == bad
    assert attn(ws=NULL) == bad and attn(ws=C.c_void_p(4096 + 16)) == bad and attn(wb=n.value - 1) == bad
    assert "workspace" in _err()
    assert attn(decay=1.5) == bad and attn(decay=float("nan")) == bad
    assert attn(decay=0.5) == bad and "weights" in _err()  # the cache has none

    def append(k=OK, ks=0, v=OK, vs=0, cache=K):
        return L.fp_cache_append(P, cache, k, ks, v, vs, NULL, NULL, NULL)
    assert append(cache=None) == bad and append(k=NULL) == bad and append(v=NULL) == bad
    assert append(k=mis) == bad and append(v=mis) == bad and append(ks=255) == bad and append(vs=260) == bad

    def select(budget=64, sinks=4, recent=8, mv=OK, cnt=OK, nl=OK, cache=K):
        return L.fp_cache_select(P, cache, budget, sinks, recent, NULL, mv, cnt, nl, NULL, NULL)
    assert select() == bad and "weights" in _err()
    c.weights = 4096
    assert select(cache=None) == bad and select(budget=0) == bad and select(budget=-3) == bad
    assert select(sinks=-1) == bad and select(recent=-1) == bad and select(sinks=60, recent=5) == bad
    assert select(sinks=1 << 30, recent=(1 << 31) - 1) == bad
    assert select(mv=NULL) == bad and select(cnt=NULL) == bad and select(nl=NULL) == bad
    assert select(mv=C.c_void_p(4100)) == bad

    def compact(budget=64, mv=OK, cnt=OK, nl=OK, cache=K):
        return L.fp_cache_compact(P, cache, budget, mv, cnt, nl, NULL, NULL)
    assert compact(cache=None) == bad and compact(budget=0) == bad and compact(mv=NULL) == bad
    assert compact(cnt=NULL) == bad and compact(nl=NULL) == bad
    c.weights = 4098
    assert select() == bad and "aligned" in _err()
    c.weights = 4096
    c.page_size = 40  # edited into an inconsistent state: refused by every call
    assert attn() == bad and append() == bad and select() == bad and compact() == bad
    c.page_size = 48
    p.head_dim = 64
    assert attn() == fp.FP_ERR_UNSUPPORTED


def test_selection_refuses_results_that_overlap_what_it_reads():
    """Other heads of a sequence still read its length and position when the first one writes its results."""
    st, p, c = _cache(lens=C.c_void_p(1 << 20))
    assert st == fp.FP_OK
    c.weights = 4096

    def select(cnt, nl, nxt=NULL):
        return fp._lib.fp_cache_select(C.byref(p), C.byref(c), 64, 4, 8, nxt, OK, C.c_void_p(cnt), C.c_void_p(nl), NULL,
                                       NULL)
    lens, nxt, far = 1 << 20, 1 << 21, 1 << 22  # 3 sequences of 2 kv-heads: 12 and 24 bytes
    for nl in (lens, lens + 8, lens - 8):
        assert select(far, nl) == fp.FP_ERR_INVALID_ARG and "overlap" in _err()
    for cnt in (lens, lens + 8, lens - 20):
        assert select(cnt, far) == fp.FP_ERR_INVALID_ARG and "overlap" in _err()
    assert select(far, nxt, C.c_void_p(nxt)) == fp.FP_ERR_INVALID_ARG and "overlap" in _err()
    assert select(nxt - 20, far, C.c_void_p(nxt)) == fp.FP_ERR_INVALID_ARG and "overlap" in _err()


def test_collected_weights_refuse_an_output_over_the_queries():
    """The weights of long pieces are summed from q after out was written."""
    st, p, c = _cache()
    assert st == fp.FP_OK
    c.weights = 4096
    n = C.c_int64(0)
    assert fp._lib.fp_cache_attn_workspace(C.byref(p), C.byref(c), C.byref(n)) == fp.FP_OK

    def attn(out, stride=0):
        return fp._lib.fp_cache_attn(C.byref(p), C.byref(c), C.c_void_p(q), stride, C.c_float(0.0), OK, n.value,
                                     C.c_void_p(out), NULL, C.c_float(0.5), NULL, NULL)
    q, row = 1 << 24, 8 * 128 * 2  # 10 tokens of 8 heads
    for out, stride in ((q, 0), (q + 9 * row, 0), (q - 9 * row, 0), (q + 9 * 2 * row, 2 * 8 * 128), (q + row, 2 * 8 * 128)):
        assert attn(out, stride) == fp.FP_ERR_INVALID_ARG and "overlap" in _err()


def test_sizes_past_two_to_the_thirty_are_refused():
    """Slot and list indices step past the last one in int32."""
    top = 1 << 30
    wide = dict(max_pages=(1 << 27) + 1, page_size=16)
    st, _, c = _cache(max_len=top, **wide)
    assert st == fp.FP_OK and c.max_len == top
    st, _, c = _cache(**wide)
    assert st == fp.FP_OK and c.max_len == top  # the room of the table is larger
    assert _cache(max_len=top + 1, **wide)[0] == fp.FP_ERR_INVALID_ARG
    st, p, c = _cache(max_len=top, **wide)
    c.weights = 4096
    P, K, L, far = C.byref(p), C.byref(c), fp._lib, C.c_void_p(1 << 40)
    for budget in (top + 1, (1 << 31) - 1):
        assert L.fp_cache_select(P, K, budget, 0, 0, NULL, far, OK, OK, NULL, NULL) == fp.FP_ERR_INVALID_ARG
        assert "budget" in _err()
        assert L.fp_cache_compact(P, K, budget, far, OK, OK, NULL, NULL) == fp.FP_ERR_INVALID_ARG and "budget" in _err()
    c.max_len = top + 1  # edited past it: refused by every call
    n = C.c_int64(0)
    assert L.fp_cache_attn_workspace(P, K, C.byref(n)) == fp.FP_ERR_INVALID_ARG
    assert L.fp_cache_append(P, K, OK, 0, OK, 0, NULL, NULL, NULL) == fp.FP_ERR_INVALID_ARG


def test_calls_without_new_tokens_need_no_tensors():
    st, p, c = _cache(cu=(0, 0, 0, 0))
    assert st == fp.FP_OK and c.max_new == 0
    assert fp._lib.fp_cache_append(C.byref(p), C.byref(c), NULL, 0, NULL, 0, NULL, NULL, NULL) == fp.FP_OK
    assert fp._lib.fp_cache_attn(C.byref(p), C.byref(c), NULL, 0, C.c_float(0), NULL, 0, NULL, NULL, C.c_float(-1.0),
                                 NULL, NULL) == fp.FP_OK


def test_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    fl = [f[0] for f in fp.fp_kv_cache._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp.h"\nint main(void) {\n'
                   + '  printf("%zu\\n", sizeof(fp_kv_cache));\n'
                   + "".join(f'  printf("%zu\\n", offsetof(fp_kv_cache, {f}));\n' for f in fl) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.check_call([cc, "-I", os.path.join(root, "include"), "-o", str(exe), str(src)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [C.sizeof(fp.fp_kv_cache)] + [getattr(fp.fp_kv_cache, f).offset for f in fl]


# ----------------------------------------------------------------------------- the Python binding
def _py(**kw):
    p = fp.Problem(np.array([0, 1, 3], np.int32), torch.zeros(3, dtype=torch.int32), 8, 2, 128, 128)
    a = dict(k_cache=torch.zeros((64, 2, 128), dtype=torch.bfloat16), lens=torch.zeros(2, dtype=torch.int32),
             block_table=torch.zeros((2, 2), dtype=torch.int32), page_size=16)
    a.update(kw)
    a.setdefault("v_cache", torch.zeros_like(a["k_cache"]))
    return p, fp.kv_cache(p, a["k_cache"], a["v_cache"], a["lens"], a["block_table"], a["page_size"],
                          a.get("weights"), a.get("positions"), a.get("max_len", 0))


@pytest.mark.parametrize("kw", [
    dict(k_cache=torch.zeros((64, 2, 128))),
    dict(k_cache=torch.zeros((64, 4, 128), dtype=torch.bfloat16)),
    dict(k_cache=torch.zeros((65, 2, 128), dtype=torch.bfloat16)),
    dict(k_cache=torch.zeros((64, 2, 256), dtype=torch.bfloat16)[..., :128]),
    dict(v_cache=torch.zeros((48, 2, 128), dtype=torch.bfloat16)),
    dict(lens=torch.zeros(3, dtype=torch.int32)), dict(lens=torch.zeros(2, dtype=torch.int64)),
    dict(block_table=torch.zeros((3, 2), dtype=torch.int32)), dict(block_table=torch.zeros((2, 2))),
    dict(block_table=torch.zeros((2, 4), dtype=torch.int32)[:, ::2]),
    dict(weights=torch.zeros(63)), dict(weights=torch.zeros(128, dtype=torch.float64)),
    dict(positions=torch.zeros(128)), dict(page_size=0),
])
def test_binding_refuses_tensors_that_do_not_fit(kw):
    with pytest.raises(ValueError):
        _py(**kw)


def test_binding_passes_on_what_the_library_refuses():
    with pytest.raises(fp.FpError):
        _py(page_size=8)
    with pytest.raises(fp.FpError):
        _py(max_len=1000)


def test_binding_checks_the_calls_tensors():
    p, c = _py(weights=torch.zeros((4, 2, 16)))
    kv = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    for k in (kv.float(), kv[:2], kv.transpose(0, 1), kv[..., ::2], torch.zeros((3, 2, 256), dtype=torch.bfloat16)[..., ::2]):
        with pytest.raises(ValueError):
            fp.cache_append(p, c, k, kv)
    with pytest.raises(ValueError):
        fp.cache_append(p, c, kv, kv, next_pos=torch.zeros(2, dtype=torch.int64))
    other = fp.Problem(np.array([0, 1, 3], np.int32), torch.zeros(3, dtype=torch.int32), 8, 2, 128, 128)
    with pytest.raises(ValueError):
        fp.cache_append(other, c, kv, kv)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)
    for out, lse, decay in ((q.float(), None, None), (q[:2], None, None), (q, torch.zeros(7), None), (q, None, 2.0),
                            (q, None, -0.5)):
        with pytest.raises(ValueError):
            fp.cache_attn(p, c, q, 0.0, ws, out, lse, decay)
    mv, cnt, nl = (torch.zeros(s, dtype=torch.int32) for s in ((2, 2, 8, 2), (2, 2), (2,)))
    for a in ((mv[:1], cnt, nl), (mv, cnt[:1], nl), (mv, cnt, cnt), (mv.float(), cnt, nl)):
        with pytest.raises(ValueError):
            fp.cache_select(p, c, 8, 0, 0, None, *a)
        with pytest.raises(ValueError):
            fp.cache_compact(p, c, 8, *a)


@pytest.mark.parametrize("heads", [1, 2, 8])
def test_binding_refuses_rows_that_overlap(heads):
    """An expanded tensor has a token stride of 0, which the C calls take for packed rows."""
    one = torch.zeros((1, heads, 128), dtype=torch.bfloat16)
    cpu = torch.device("cpu")
    flat = torch.zeros(64 * heads * 128, dtype=torch.bfloat16)
    for t in (one.expand(64, heads, 128), flat.as_strided((64, heads, 128), (heads * 128 - 8, 128, 1))):
        with pytest.raises(ValueError, match="overlap"):
            fp._rows_of(t, "q", 64, heads, 128, cpu)
    # a single token has no neighbour; rows further apart than packed are a slice of a wider projection
    assert fp._rows_of(one, "q", 1, heads, 128, cpu) == (one.data_ptr(), 0)
    wide = torch.zeros((64, heads + 3, 128), dtype=torch.bfloat16)
    assert fp._rows_of(wide[:, 1:1 + heads], "q", 64, heads, 128, cpu) == (wide.data_ptr() + 256, (heads + 3) * 128)
    # and through the calls themselves
    p, c = _py()
    kv, q = torch.zeros((3, 2, 128), dtype=torch.bfloat16), torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    for k, v in ((kv[:1].expand(3, 2, 128), kv), (kv, kv[:1].expand(3, 2, 128))):
        with pytest.raises(ValueError, match="overlap"):
            fp.cache_append(p, c, k, v)
    with pytest.raises(ValueError, match="overlap"):
        fp.cache_attn(p, c, q[:1].expand(3, 8, 128), 0.0, torch.zeros(16, dtype=torch.uint8), q)
