"""Pins of the paged-cache oracle (oracle/pages.py) and the bounds of the cache's index arithmetic
(csrc/pages_index.h, compiled here as plain C++).  CPU only."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import flow_matching_action_expert_b200 as R
from flow_matching_action_expert_b200 import build as B
from oracle import pages as OP

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _empty_cache(batch, width, n_pages):
    rng = np.random.default_rng(3)
    return np.full((batch, width), -1, np.int32), rng.permutation(n_pages).astype(np.int32)


def test_plan_hands_out_every_page_once_and_takes_them_back():
    page, n_pages, batch, width = 4, 40, 6, 12
    rng = np.random.default_rng(5)
    table, free = _empty_cache(batch, width, n_pages)
    lens, nf = np.zeros(batch, np.int32), n_pages
    for _ in range(60):
        delta = np.array([rng.integers(-12, 14) for _ in range(batch)])
        r = OP.plan(lens, delta, table, free, nf, page, n_pages, 200)
        table, free, nf, lens = r["table"], r["free"], r["n_free"], r["lens"]
        held = [table[b, i] for b in range(batch) for i in range(OP.pages_for(lens[b], page))]
        assert sorted(held + list(free[:nf])) == list(range(n_pages))
        live = r["slots"][r["slots"] >= 0]
        assert len(set(live)) == len(live)
    r = OP.plan(lens, [-10 ** 9] * batch, table, free, nf, page, n_pages, 0)
    assert r["n_free"] == n_pages and not r["lens"].any() and sorted(r["free"]) == list(range(n_pages))


def test_plan_rows_follow_the_request_and_refusals_leave_it():
    table, free = _empty_cache(3, 8, 5)
    r = OP.plan([0, 0, 0], [5, 12, 3], table, free, 5, 4, 5, 24)
    # 2 + 3 pages fit; the third request needs one more and is refused
    assert list(r["lens"]) == [5, 12, 0] and r["err"] == {"no_pages"} and r["n_free"] == 0
    assert list(r["row_start"]) == [0, 5, 17, 20] and (r["slots"][17:] == -1).all()
    assert list(r["positions"][:17]) == list(range(5)) + list(range(12))
    assert r["slots"][4] == r["table"][0, 1] * 4
    r = OP.plan([0, 0, 0], [5, 33, 3], table, free, 5, 4, 5, 41)
    assert list(r["lens"]) == [5, 0, 3] and r["err"] == {"bounds"}


def test_attention_matches_torch_on_shuffled_pages():
    rng = np.random.default_rng(7)
    page, n_pages, hkv, d, n, G = 8, 12, 2, 64, 61, 3
    k, v = rng.normal(size=(2, n_pages, hkv, page, d))
    row = rng.permutation(n_pages)[:8]
    q = rng.normal(size=(G, d))
    for h in range(hkv):
        out, size, _ = OP.attend_one(q, OP.keys_of(k, row, n, h, page), OP.keys_of(v, row, n, h, page))
        flat = [torch.from_numpy(x[row][:, h].reshape(-1, d)[:n].copy()) for x in (k, v)]
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q)[None], flat[0][None], flat[1][None])
        assert np.abs(out - ref[0].numpy()).max() < 1e-12 and (size >= np.abs(out) - 1e-12).all()
    assert not OP.attend_one(q, np.zeros((0, d)), np.zeros((0, d)))[0].any()


@pytest.mark.parametrize("mistake", ["last key missing", "one key too many", "scale", "heads swapped",
                                     "page off by one", "value of the next key"])
@pytest.mark.parametrize("u, f16", [(2.0 ** -8, False), (2.0 ** -11, True)])
def test_planted_mistakes_leave_the_attention_tolerance(mistake, u, f16):
    """Each mistake, made in the oracle, lands outside the bound the GPU tests use on 200 keys."""
    from pages_tolerances import attend_tolerance
    rng = np.random.default_rng(17)
    d, n, page, G = 128, 200, 16, 4
    k, v = rng.normal(size=(2, 20, 1, page, d))
    row, q = rng.permutation(20)[:13], rng.normal(size=(G, d))
    kk, vv = OP.keys_of(k, row, n, 0, page), OP.keys_of(v, row, n, 0, page)
    ref, size, big = OP.attend_one(q, kk, vv)
    if mistake == "last key missing":
        bad = OP.attend_one(q, kk[:-1], vv[:-1])[0]
    elif mistake == "one key too many":
        bad = OP.attend_one(q, OP.keys_of(k, row, n + 1, 0, page), OP.keys_of(v, row, n + 1, 0, page))[0]
    elif mistake == "scale":
        bad = OP.attend_one(q * d ** -0.5, kk, vv)[0]
    elif mistake == "heads swapped":
        bad = OP.attend_one(q[::-1], kk, vv)[0]
    elif mistake == "page off by one":
        bad = OP.attend_one(q, OP.keys_of(k, (row + 1) % 20, n, 0, page), vv)[0]
    else:
        bad = OP.attend_one(q, kk, np.roll(vv, -1, 0))[0]
    tol = attend_tolerance(u, d, f16, ref, size, big, vv)
    assert (np.abs(bad - ref) > tol).mean() > 0.1


def test_rope_is_the_prefix_models_rotation():
    from oracle import model as O
    x = np.random.default_rng(9).normal(size=(5, 256))
    pos = np.array([0, 1, 255, 256, 5000])
    got = np.stack([OP.rope(x[t], int(pos[t]), 10000.0) for t in range(5)])
    assert np.abs(got - O.rope(x, pos, 10000.0)).max() < 1e-10


def test_prefix_step_is_the_prefix_pass_of_the_last_token():
    """Layer 0's keys and values do not depend on the mask, so the last of n tokens gets from a step
    what it gets from the whole pass: its keys of layer 1 and, alone in its cache, everything."""
    from oracle import model as O
    from synth import workloads as WL
    shape = WL.PrefillShape(n_layers=2, width=64, mlp_dim=96, n_q_heads=4, n_kv_heads=1, head_dim=16)
    W = {k: v * 8 for k, v in WL.as_f32(WL.prefill_weights(shape)).items()}
    x = np.random.default_rng(13).normal(size=(1, 7, 64)) * 8
    K, V, _ = O.prefill(W, shape, x, np.ones((1, 7), np.uint8))
    _, k, v = OP.prefix_step(W, shape, x[0, 6], K[:, 0, :6], V[:, 0, :6], 6)
    assert np.abs(k - K[:, 0, 6]).max() < 1e-11 and np.abs(v - V[:, 0, 6]).max() < 1e-11
    K, V, _ = O.prefill(W, shape, x[:, :1], np.ones((1, 1), np.uint8))
    _, k, v = OP.prefix_step(W, shape, x[0, 0], np.zeros((2, 0, 16)), np.zeros((2, 0, 16)), 0)
    assert np.abs(k - K[:, 0, 0]).max() < 1e-11 and np.abs(v - V[:, 0, 0]).max() < 1e-11


def test_choice_keeps_first_and_last_and_breaks_ties_low():
    s = np.array([9., 1., 5., 5., 5., 2., 8., 0.])
    assert OP.choose(s, 8, 8, 1, 1) == list(range(8))
    assert OP.choose(s, 8, 4, 1, 1) == [0, 2, 6, 7]
    assert OP.choose(s, 8, 5, 1, 1) == [0, 2, 3, 6, 7]
    assert OP.choose(s, 8, 3, 1, 2) == [0, 6, 7]


@pytest.fixture(scope="module")
def index_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("pg")
    src = d / "t.cc"
    src.write_text('''
#include <stddef.h>
#include "pages_index.h"
using namespace rtvla;
extern "C" {
int key_row(const int *row, const int *sel, int j, int n, int len, int shift, int pages, int width, int *bad) {
  PageGeom g{shift, pages, width, 1, 64}; bool b = false;
  int r = pg_key_row(row, sel, j, n, len, g, &b); *bad = b; return r; }
int list_len(int len, int n_sel, int listed, int shift, int pages, int width) {
  PageGeom g{shift, pages, width, 1, 64}; return pg_list_len(len, n_sel, listed, g); }
int clamp_len(int len, int shift, int pages, int width, int *bad) {
  PageGeom g{shift, pages, width, 1, 64}; bool b = false; int r = pg_len(len, g, &b); *bad = b; return r; }
int slot(int s, int shift, int pages, int *bad) {
  PageGeom g{shift, pages, 1, 1, 64}; bool b = false; int r = pg_slot(s, g, &b); *bad = b; return r; }
size_t elem(int layer, int row, int h, int shift, int pages, int heads, int d) {
  PageGeom g{shift, pages, 1, heads, d}; return pg_elem(layer, row, h, g); }
}''')
    so = d / "t.so"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, "-o", str(so), str(src)])
    lib = ctypes.CDLL(str(so))
    lib.elem.restype = ctypes.c_size_t
    return lib


WILD = (-2 ** 31, -1000, -2, -1, 0, 1, 4, 5, 6, 7, 8, 63, 64, 1000, 2 ** 31 - 1)


def test_bad_lengths_pages_and_slots_never_leave_the_pool(index_lib):
    bad = ctypes.c_int()
    for shift, pages, width in ((0, 5, 3), (2, 7, 4), (4, 8, 2)):
        cap = width << shift
        for len_ in WILD:
            n = index_lib.clamp_len(len_, shift, pages, width, ctypes.byref(bad))
            assert 0 <= n <= cap and bool(bad.value) == (not 0 <= len_ <= cap)
        for s in WILD:
            r = index_lib.slot(s, shift, pages, ctypes.byref(bad))
            ok = 0 <= s < pages << shift
            assert r == (s if ok else -1) and bool(bad.value) == (not ok and s != -1)
        for entry in WILD:
            for len_ in range(cap + 1):
                row = (ctypes.c_int * width)(*([entry] * width))
                for chosen in (None,) + WILD:
                    n_sel = 3
                    sel = (ctypes.c_int * n_sel)(*([chosen] * n_sel)) if chosen is not None else None
                    n = index_lib.list_len(len_, n_sel, int(sel is not None), shift, pages, width)
                    assert 0 <= n <= (cap if sel is None else n_sel << shift)
                    for j in sorted({-1, 0, 1, n // 2, max(n - 1, 0), n, n + 1}):
                        r = index_lib.key_row(row, sel, j, n, len_, shift, pages, width, ctypes.byref(bad))
                        assert -1 <= r < pages << shift
                        if r >= 0:
                            assert r >> shift == entry and not bad.value
                        elif 0 <= j < n and sel is None:
                            assert bad.value


def test_element_offsets_pass_32_bits(index_lib):
    # layer 17 of a pool of 2^20 pages of 64 tokens, 1 head of 256
    want = (((17 * 2 ** 20 + 1048575) * 64) + 63) * 256
    assert index_lib.elem(17, 2 ** 26 - 1, 0, 6, 2 ** 20, 1, 256) == want > 2 ** 32


def _cfg(**kw):
    args = dict(n_pages=8, table_width=4)
    args.update(kw)
    return R.make_pages_config(**args)


@pytest.mark.parametrize("kw, name", [
    (dict(n_pages=0), "INVALID_ARG"), (dict(table_width=0), "INVALID_ARG"), (dict(max_batch=0), "INVALID_ARG"),
    (dict(max_batch=4097), "INVALID_ARG"), (dict(n_q_heads=9, n_kv_heads=2), "INVALID_ARG"),
    (dict(n_pages=2 ** 27, page_size=16), "INVALID_ARG"), (dict(table_width=2 ** 20 + 1), "INVALID_ARG"),
    (dict(rope_theta=-1.0), "INVALID_ARG"), (dict(rope_theta=float("inf")), "INVALID_ARG"),
    (dict(n_layers=0), "INVALID_ARG"), (dict(dtype=2), "UNSUPPORTED"), (dict(head_dim=72), "UNSUPPORTED"),
    (dict(n_q_heads=17, n_kv_heads=1), "UNSUPPORTED"), (dict(page_size=24), "UNSUPPORTED"),
    (dict(page_size=2048, table_width=1), "UNSUPPORTED")])
def test_shapes_are_refused_before_any_cuda_call(kw, name):
    B.build()
    with pytest.raises(R.RtvlaError) as e:
        R.rtvla_pages_create(_cfg(**kw))
    assert e.value.name == "RTVLA_ERR_" + name


def test_null_arguments_are_refused():
    B.build()
    lib = R.library()
    kv = R.make_paged_kv(None, None, None, None, None, 1)
    ref = ctypes.byref(kv)
    for code in (lib.rtvla_pages_plan(None, None, None, None, None, ref, None, None, None, None, 0, None),
                 lib.rtvla_pages_write(None, 0, None, 0, None, None, 0, ref, None, None),
                 lib.rtvla_pages_attend(None, 0, None, ref, None, 0, None, None),
                 lib.rtvla_pages_select(None, 0, None, ref, 1, 0, 1, None, None),
                 lib.rtvla_prefix_step(None, None, None, None, None, ref, None, None),
                 lib.rtvla_pages_sync_status(None, None)):
        assert R.STATUS[code] == "RTVLA_ERR_INVALID_ARG"
    R.rtvla_pages_destroy(0)
    assert "free list" in R.rtvla_status_string(10)
