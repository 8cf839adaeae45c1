"""The paged KV cache where one wrong step would hide at ordinary values: infinities, weights far below
the maximum, page lists and bad pages in the split attention, many rows in one write, scores whose
partial sums overflow.  Against the fp64 oracle.

Tolerances: tests/pages_tolerances.py, without its term for small f16 weights (weight_tolerance).
"""
import numpy as np
import pytest
import torch

import flow_matching_action_expert_b200 as R
from oracle import pages as OP

from pages_tolerances import E32
from test_gpu_pages import Cache, check_select, i32, run_plan

pytestmark = pytest.mark.gpu


def weight_tolerance(u, d, f16, ref, size, big, vv):
    """As attend_tolerance, but an f16 weight p counts within 2^-22 p + 2^-40 of the largest: two parts of
    11 bits (2^-11 * 2^-11), the first of the weight times 2^15, so that half a step of the smallest
    numbers, 2^-25, is 2^-40.  (bf16: two parts of 8 bits, 2^-16 p, no smallest step that matters.)"""
    n = len(vv)
    tol = u * np.abs(ref) + (2 * (d + 4) * E32 * big + (2 * n + 136) * E32 + 2.0 ** (-22 if f16 else -16)) * size
    if f16:
        tol = tol + 2.0 ** -25 + n * 2.0 ** -40 * (np.abs(vv).max() if n else 0.0)
    return tol


class Tight(Cache):
    def close(self, got, ref, size, big, kk, vv, what):
        tol = weight_tolerance(self.u, self.d, self.f16, ref, size, big, vv)
        err = np.abs(got - ref)
        assert np.isfinite(got).all() and (err <= tol).all(), (what, float((err - tol).max()))
        if len(kk) == 0:
            assert not got.any()


ROOMS = [None, 8192]  # table rows with room for 8192 tokens make one request go to the split attention


def roomy(room, page):
    return room and OP.pages_for(room, page)


# ---------------------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("nats", [12.0, 16.0, 18.0, 22.0])
def test_attend_long_tail_of_small_weights(dtype, room, nats):
    """One dominant key in every 16, the others `nats` below it (18: 2^-26), which alone have values: their
    sum, 15000 e^-nats, is what the output is made of."""
    c = Tight([1024], dtype, hq=1, d=64, width=roomy(room, 16))
    at = torch.zeros((1024, 64), dtype=c.t, device="cuda")
    at[:, 0] = -nats
    at[::16, 0] = 0.0
    pages = c.table[0, :64].long()
    c.k[0, pages, 0] = at.view(64, 16, 64)
    at[:] = 1000.0
    at[::16] = 0.0
    c.v[0, pages, 0] = at.view(64, 16, 64)
    c.q.zero_()
    c.q[0, 0, 0] = 8.0  # logits are the keys' first component
    c.check_attend(c.attend())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq, hkv, d", [(8, 1, 256), (16, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("std", [1.0, 3.0])
def test_attend_to_the_weights_own_precision(dtype, hq, hkv, d, room, std):
    c = Tight([1000, 17, 333], dtype, hq, hkv, d, width=roomy(room, 16), std=std)
    c.check_attend(c.attend())


def _lists(c, width, rng):
    """Lists of `width` of a request's pages in any order, some twice; -1 past the pages held."""
    B = len(c.lens_np)
    sel, picks = np.full((B, c.hkv, width), -1, np.int32), [[None] * c.hkv for _ in range(B)]
    for b, n in enumerate(c.lens_np):
        held = OP.pages_for(int(n), c.page)
        m = min(width, held)
        for h in range(c.hkv):
            pick = list(rng.integers(0, held, m)) if m else []
            if m and h % 2 == 0:
                pick[0] = held - 1  # the last page, not full, in front
            sel[b, h, :m], picks[b][h] = pick, pick
    return sel, picks


# batches beyond the clusters' share of the GPU, and one request with a list too long for a cluster
SPLIT = [dict(lens=[700 + 7 * i for i in range(40)] + [0, 1, 33], hq=8, hkv=2, d=64, page=16, sel_width=40),
         dict(lens=[9001], hq=8, hkv=1, d=256, page=64, sel_width=64),
         dict(lens=[5000, 0, 4999], hq=12, hkv=1, d=128, page=32, sel_width=128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", SPLIT)
def test_split_attention_over_lists(dtype, case):
    case = dict(case)
    width = case.pop("sel_width")
    c = Tight(case.pop("lens"), dtype, layers=2, **case)
    sel, picks = _lists(c, width, np.random.default_rng(23))
    c.check_attend(c.attend(1, i32(sel)), 1, picks)


@pytest.mark.parametrize("case", SPLIT)
def test_split_attention_leaves_out_bad_pages_and_reports_them(case):
    case = dict(case)
    width = case.pop("sel_width")
    c = Tight(case.pop("lens"), **case)
    rng = np.random.default_rng(29)
    # every third page of a request's table is none; the last request has none at all
    bad = c.table_np.copy()
    for b, n in enumerate(c.lens_np):
        held = OP.pages_for(int(n), c.page)
        bad[b, 1:held:3] = rng.choice([-1, c.n_pages, 2 ** 31 - 1, -2 ** 31], len(range(1, held, 3)))
    last = int(np.argmax(c.lens_np))
    if len(c.lens_np) > 1:
        bad[last] = -1
    c.table.copy_(i32(bad))
    ok = [[[e for e in range(OP.pages_for(int(n), c.page)) if 0 <= bad[b, e] < c.n_pages]] * c.hkv
          for b, n in enumerate(c.lens_np)]
    c.check_attend(c.attend(status="RTVLA_ERR_DEVICE_BOUNDS"), picks=ok)
    # lists with entries that are no page of the request, over the same table
    sel, picks = _lists(c, width, rng)
    for b, n in enumerate(c.lens_np):
        held = OP.pages_for(int(n), c.page)
        for h in range(c.hkv):
            m = min(width, held)
            sel[b, h, 2:m:5] = rng.choice([-1, held, 2 ** 30], len(range(2, m, 5)))
            picks[b][h] = [int(e) for e in sel[b, h, :m] if 0 <= e < held and 0 <= bad[b, e] < c.n_pages]
    c.check_attend(c.attend(sel=i32(sel), status="RTVLA_ERR_DEVICE_BOUNDS"), picks=picks)
    c.table.copy_(i32(c.table_np))
    sel, picks = _lists(c, width, rng)
    c.check_attend(c.attend(sel=i32(sel)), picks=picks)


def test_split_attention_clamps_bad_lengths():
    c = Tight([800] * 40, hq=8, hkv=2, d=64, page=16)
    cap = c.width * 16
    lens = c.lens_np.copy()
    lens[[0, 5, 39]] = [-3, 10 ** 9, -2 ** 31]
    c.table_np[5, 50:] = c.table_np[5, :c.width - 50]  # what the clamped length reaches
    c.table.copy_(i32(c.table_np))
    c.lens.copy_(i32(lens))
    lens[[0, 5, 39]] = [0, cap, 0]
    c.check_attend(c.attend(status="RTVLA_ERR_DEVICE_BOUNDS"), lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("room", ROOMS)
def test_attend_with_infinities(dtype, room):
    """Logits of -inf have weight 0, of +inf or NaN make their head NaN, values that are not finite make
    their component so; nothing else changes."""
    inf = float("inf")
    c = Tight([500, 40, 300, 300], dtype, hq=4, hkv=1, d=64, width=roomy(room, 16))
    c.q[:, :, 0] = torch.tensor([1.0, 0.5, 2.0, -1.0], device="cuda", dtype=c.t)
    gone = [3, 16, 17, 18, 19, 200, 499]
    page, off = [int(c.table_np[0, j // 16]) for j in gone], [j % 16 for j in gone]
    c.k[0, page, 0, off, 0] = -inf                          # -inf for heads 0 to 2, +inf for head 3
    c.k[0, c.table[1, :3].long(), 0, :, 0] = -inf           # every key of the second request
    p = int(c.table_np[2, 7])
    c.v[0, p, 0, 5, 9], c.v[0, p, 0, 6, 11], c.v[0, p, 0, 7, 13] = inf, -inf, float("nan")
    c.k[0, int(c.table_np[3, 2]), 0, 1, 30] = float("nan")
    out = c.attend().double().cpu().numpy()
    k, v, q = (x.double().cpu().numpy() for x in (c.k[0], c.v[0], c.q))
    keep = [j for j in range(500) if j not in gone]
    kk, vv = (OP.keys_of(x, c.table_np[0], 500, 0, 16)[keep] for x in (k, v))
    ref, size, big = OP.attend_one(q[0, :3], kk, vv)
    assert (np.abs(out[0, :3] - ref) <= weight_tolerance(c.u, 64, c.f16, ref, size, big, vv)).all()
    assert np.isnan(out[0, 3]).all()
    assert not out[1, :3].any() and np.isnan(out[1, 3]).all()
    off = [9, 11, 13]
    rest = [i for i in range(64) if i not in off]
    kk, vv = (OP.keys_of(x, c.table_np[2], 300, 0, 16) for x in (k, v))
    ref, size, big = OP.attend_one(q[2], kk, vv[:, rest])
    assert (np.abs(out[2][:, rest] - ref) <= weight_tolerance(c.u, 64, c.f16, ref, size, big, vv[:, rest])).all()
    assert not np.isfinite(out[2][:, off]).any()
    assert np.isnan(out[3]).all()


@pytest.mark.parametrize("room", ROOMS)
def test_attend_with_a_queries_infinity(room):
    c = Tight([100, 100], hq=2, d=64, width=roomy(room, 16))
    c.q[0, 1, 4] = float("inf")
    out = c.attend()
    assert out[0, 1].isnan().all()
    c.q[0, 1] = 0.0
    clean = c.attend()
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("dtype, hq, d, lens, width", [
    ("bf16", 8, 256, [544], None), ("bf16", 8, 256, [544], 512), ("f16", 16, 64, [800] * 16, None),
    ("bf16", 8, 256, [30000, 1, 512, 9000], None)])
def test_equal_bits_beside_other_work(dtype, hq, d, lens, width):
    """Forty calls give the same bits while another stream keeps the GPU busy."""
    c = Cache(lens, dtype, hq, 1, d, width=width)
    first, busy = c.attend(), torch.cuda.Stream()
    x = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    outs = [torch.zeros_like(first) for _ in range(40)]
    with torch.cuda.stream(busy):
        for _ in range(10):
            x @ x
    for o in outs:
        R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("room", ROOMS)
def test_captured_behind_copies_and_other_streams(room):
    """A captured attention whose predecessor in the graph is a copy, a fill, or work joined from another
    stream; first in its graph; and directly behind another attention."""
    c = Cache([700, 0, 90], hq=8, d=128, width=roomy(room, 16))
    src, other = c.q.clone(), torch.randn_like(c.q)
    outs = [torch.full_like(c.q, 3.0) for _ in range(4)]
    main, fork = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, outs[0], main)
        c.q.copy_(other)
        R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, outs[1], main)
        fork.wait_stream(main)
        with torch.cuda.stream(fork):
            c.q.copy_(src)
        main.wait_stream(fork)
        R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, outs[2], main)
        R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, outs[3], main)
    for _ in range(5):
        for o in outs:
            o.fill_(3.0)
        graph.replay()
        assert c.status() == "RTVLA_OK"
        for i, o in enumerate(outs):
            c.q.copy_(other if i == 1 else src)
            c.check_attend(o)


# ---------------------------------------------------------------------------------------
# selection

def test_select_with_partial_sums_that_overflow():
    """Scores that are ordinary numbers but whose fp32 sums pass through infinity."""
    c = Cache([16 * 200], page=16, d=64, hq=1)
    c.q.fill_(1.0)
    m = c.k_mean[0, :, 0]
    pages = c.table[0].long()
    big = torch.zeros((3, 8, 8), device="cuda")   # eight components to a block
    big[0, [0, 4]], big[0, [1, 5]] = 4e37, -4e37   # + and - infinity on the way; the score is 0
    big[1, 0], big[1, 4] = -4e37, -4e37            # -infinity on the way; the score is 2e37 or so
    big[1, [1, 3]], big[1, 2] = 2.06e37, 4.12e37
    big[2, [0, 4]], big[2, [1, 3]], big[2, 2] = 4e37, -2.06e37, -4.12e37  # +infinity; the score is -2e37 or so
    m[pages[[20, 60, 110]]] = big.view(3, 64).to(c.t)
    for budget in (2, 30, 199):
        sel = torch.empty((1, 1, budget), dtype=torch.int32, device="cuda")
        R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, budget, 0, 1, sel)
        assert c.status() == "RTVLA_OK"
        check_select(c, sel, budget, 0, 1)


# ---------------------------------------------------------------------------------------
# plan and write

def test_plan_reports_a_bad_page_given_back():
    c = Cache([40, 64], d=64, hq=1, page=16)
    c.table_np[0, 2] = c.n_pages + 3
    assert "bounds" in run_plan(c, [40, 64], [-20, 0], 4)["err"]
    c.table_np[0, 2] = -1
    assert "bounds" in run_plan(c, [40, 64], [-40, 0], 4)["err"]
    assert not run_plan(c, [40, 64], [-7, 0], 4)["err"]  # the request keeps it


def _write_long(c, lens, new, pad, src, layer=0):
    ref = OP.plan(lens, new, c.table_np, c.free_np, c.n_free, c.page, c.n_pages, int(sum(new)))
    assert not ref["err"]
    rng = np.random.default_rng(31)
    T = int(sum(new)) + pad
    # skipped rows only between requests: a page's rows follow one another
    req = np.repeat(np.arange(len(new)), new)
    gap = np.sort(rng.choice(len(new) + 1, pad)) if pad else np.zeros(0, int)
    at = np.arange(T - pad) + np.searchsorted(gap, req, side="right")
    slots, pos = np.full(T, -1, np.int32), np.zeros(T, np.int32)
    slots[at], pos[at] = ref["slots"], ref["positions"]
    qkv = torch.randn((T, (c.hq + 2 * c.hkv) * c.d), device="cuda")
    qkv = qkv if src == "f32" else qkv.to(c.t)
    code = R.DTYPE_F32 if src == "f32" else c.cfg.dtype
    q_out = torch.full((T, c.hq, c.d), 555.0, dtype=c.t, device="cuda")
    before = c.k_mean.clone()
    R.rtvla_pages_write(c.ctx, layer, qkv, code, i32(slots), i32(pos), T, c.kv, q_out)
    assert c.status() == "RTVLA_OK"
    return slots, pos, qkv, q_out, before


@pytest.mark.parametrize("dtype, src, hq, hkv, page, lens, new, pad", [
    # a CTA looks for full pages in 16 rows, in 64, in 256, in 512
    ("bf16", "f32", 1, 1, 2, [0, 5, 100, 63], [1500, 1, 1409, 90], 1),
    ("f16", "same", 4, 4, 16, [7, 0, 300], [1000, 17, 2002], 40),
    ("bf16", "same", 4, 4, 4, [3, 0, 17, 1], [5003, 1, 4000, 3300], 57),
    ("f16", "f32", 8, 8, 1, [0, 9], [9000, 3001], 3),
    ("bf16", "f32", 2, 2, 128, [100, 1], [11000, 127], 0)])
def test_write_of_thousands_of_rows(dtype, src, hq, hkv, page, lens, new, pad):
    need = sum(OP.pages_for(n + m, page) - OP.pages_for(n, page) for n, m in zip(lens, new))
    c = Cache(lens, dtype, hq, hkv, 64, page, width=OP.pages_for(12000, page), spare=need + 3)
    slots, pos, qkv, q_out, before = _write_long(c, lens, new, pad, src)
    live = torch.from_numpy(slots >= 0).cuda()
    sl = torch.from_numpy(slots[slots >= 0].astype(np.int64)).cuda()
    full = sl[sl % page == page - 1] // page
    stored = c.k[0, full].double()
    ref, got = stored.mean(2), c.k_mean[0, full].double()
    tol = c.u * ref.abs() + page * E32 * stored.abs().mean(2) + (2.0 ** -25 if c.f16 else 0.0)
    assert len(full) and ((got - ref).abs() <= tol).all()
    before[0, full] = c.k_mean[0, full]
    assert torch.equal(c.k_mean.view(torch.int16), before.view(torch.int16))  # no other page's mean
    # rows against the formula, in fp64 on the GPU
    x = qkv.double().view(len(slots), hq + 2 * hkv, 64)
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    ang = torch.from_numpy(pos).cuda().double()[:, None, None] * freq
    x1, x2 = x[:, :hq + hkv, :32], x[:, :hq + hkv, 32:]
    y = torch.cat((x1 * ang.cos() - x2 * ang.sin(), x2 * ang.cos() + x1 * ang.sin()), -1)
    tol = 8 * E32 * torch.cat([x1.abs() + x2.abs()] * 2, -1) + c.u * y.abs() + (2.0 ** -25 if c.f16 else 0.0)
    assert ((q_out.double() - y[:, :hq]).abs() <= tol[:, :hq])[live].all()
    assert (q_out[~live] == float(torch.tensor(555.0).to(c.t))).all()
    k, v = (t[0, sl // page, :, sl % page] for t in (c.k, c.v))
    assert ((k.double() - y[live, hq:]).abs() <= tol[live, hq:]).all()
    assert torch.equal(v, x[live, hq + hkv:].to(c.t))


@pytest.mark.parametrize("page, bad_row", [(4, 1), (16, 0), (16, 14)])
def test_mean_of_a_page_with_a_skipped_row(page, bad_row):
    """A row whose position is none is skipped; its page's mean is of the key that is stored there."""
    c = Cache([2 * page], d=64, hq=1, page=page, width=4)
    p = int(c.table_np[0, 1])
    slots, pos = p * page + np.arange(page), page + np.arange(page)
    pos[bad_row] = -5 if bad_row else 4 * page
    q_out = torch.zeros((page, 1, 64), dtype=c.t, device="cuda")
    kept = c.k[0, p, 0, bad_row].clone()
    R.rtvla_pages_write(c.ctx, 0, torch.randn((page, 192), device="cuda"), R.DTYPE_F32, i32(slots), i32(pos), page,
                        c.kv, q_out)
    assert c.status() == "RTVLA_ERR_DEVICE_BOUNDS"
    assert torch.equal(c.k[0, p, 0, bad_row], kept)
    stored = c.k[0, p, 0].double()
    ref = stored.mean(0)
    assert ((c.k_mean[0, p, 0].double() - ref).abs()
            <= c.u * ref.abs() + page * E32 * stored.abs().mean(0)).all()
