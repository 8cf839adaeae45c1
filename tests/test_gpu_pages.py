"""The paged KV cache on the GPU (rtvla_pages_*), against the fp64 oracle.

Tolerances: tests/pages_tolerances.py.  Plans and selections are equal.
"""
import numpy as np
import pytest
import torch

import flow_matching_action_expert_b200 as R
from oracle import pages as OP

from pages_tolerances import E32, attend_tolerance

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, R.DTYPE_BF16), "f16": (torch.float16, R.DTYPE_F16)}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """A context, a pool with shuffled pages, NaN in every slot no request holds."""

    def __init__(self, lens, dtype="bf16", hq=8, hkv=1, d=256, page=16, layers=1, width=None, seed=1, theta=10000.0,
                 spare=5, std=1.0, **kw):
        self.t, code = TYPES[dtype]
        self.u = torch.finfo(self.t).eps / 2
        self.f16 = dtype == "f16"
        self.hq, self.hkv, self.d, self.page, self.layers, self.theta = hq, hkv, d, page, layers, theta
        self.lens_np = np.array(lens, np.int32)
        held = [OP.pages_for(n, page) for n in lens]
        self.width = width or max(held + [1]) + 2
        self.n_pages = sum(held) + spare
        rng = np.random.default_rng(seed)
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table_np = np.full((len(lens), self.width), -7, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table_np[b, :n] = order[at:at + n]
            at += n
        self.free_np = np.concatenate([order[at:], np.full(at, -9, np.int32)])
        self.n_free = self.n_pages - at
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (layers, self.n_pages, hkv, page, d)
        self.k = (torch.randn(shape, generator=g, device="cuda") * std).to(self.t)
        self.v = torch.randn(shape, generator=g, device="cuda").to(self.t)
        dead = np.ones((self.n_pages, page), bool)
        for b, n in enumerate(lens):
            for t in range(n):
                dead[self.table_np[b, t // page], t % page] = False
        for x in (self.k, self.v):
            x.masked_fill_(torch.from_numpy(dead).cuda()[None, :, None, :, None], float("nan"))
        self.k_mean = self.k.float().mean(3).to(self.t)
        self.table, self.lens = i32(self.table_np), i32(self.lens_np)
        self.cfg = R.make_pages_config(n_pages=self.n_pages, table_width=self.width, page_size=page, dtype=code,
                                       n_layers=layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                                       max_batch=len(lens), rope_theta=theta, **kw)
        self.ctx = R.rtvla_pages_create(self.cfg)
        self.kv = R.make_paged_kv(self.k, self.v, self.k_mean, self.table, self.lens, len(lens))
        self.q = (torch.randn((len(lens), hq, d), generator=g, device="cuda") * std).to(self.t)

    def __del__(self):
        if getattr(self, "ctx", 0) and R is not None and R.rtvla_pages_destroy is not None:
            R.rtvla_pages_destroy(self.ctx)

    def status(self):
        return R.STATUS[R.rtvla_pages_sync_status(self.ctx)]

    def attend(self, layer=0, sel=None, status="RTVLA_OK"):
        out = torch.full_like(self.q, 777.0)
        R.rtvla_pages_attend(self.ctx, layer, self.q, self.kv, sel, sel.shape[-1] if sel is not None else 0, out)
        assert self.status() == status
        return out

    def check_attend(self, out, layer=0, picks=None, lens=None, rows=None):
        """picks[b][h]: lists of logical pages, None for all."""
        k, v = self.k[layer].float().cpu().numpy(), self.v[layer].float().cpu().numpy()
        q, got = self.q.double().cpu().numpy(), out.double().cpu().numpy()
        G = self.hq // self.hkv
        for b in range(len(self.lens_np)) if rows is None else rows:
            n = int((self.lens_np if lens is None else lens)[b])
            for h in range(self.hkv):
                pick = picks[b][h] if picks is not None else None
                kk, vv = (OP.keys_of(x, self.table_np[b], n, h, self.page, pick) for x in (k, v))
                ref, size, big = OP.attend_one(q[b, h * G:(h + 1) * G], kk, vv)
                self.close(got[b, h * G:(h + 1) * G], ref, size, big, kk, vv, (b, h, n))

    def close(self, got, ref, size, big, kk, vv, what):
        tol = attend_tolerance(self.u, self.d, self.f16, ref, size, big, vv)
        err = np.abs(got - ref)
        assert np.isfinite(got).all() and (err <= tol).all(), (what, float((err - tol).max()))
        if len(kk) == 0:
            assert not got.any()


EDGE = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 0, 333]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq, hkv, d, page", [(8, 1, 256, 16), (1, 1, 256, 64), (16, 1, 256, 1), (8, 8, 128, 32),
                                              (14, 2, 128, 8), (9, 3, 64, 256), (32, 2, 64, 2), (7, 1, 64, 1024)])
@pytest.mark.parametrize("room", [None, 8192])  # tokens a table row has room for: it decides how work is split
def test_attend_over_edge_lengths(dtype, hq, hkv, d, page, room):
    c = Cache(EDGE, dtype, hq, hkv, d, page, layers=2, width=room and OP.pages_for(room, page))
    for layer in (1, 0):
        c.check_attend(c.attend(layer), layer)


@pytest.mark.parametrize("lens", [[20011], [4096, 1, 0, 3000], [0], [1], [0] * 9, list(range(1, 401)), [65] * 700,
                                  [0] * 150 + [5000] + [0] * 150, [16384, 16384]])
def test_attend_over_batches_and_lengths(lens):
    c = Cache(lens, d=64, page=16)
    c.check_attend(c.attend())


@pytest.mark.parametrize("std", [0.0, 4.0])
def test_attend_flat_and_peaked_softmax(std):
    # std 0: equal keys, the mean of the values; std 4: one key takes nearly all the weight
    c = Cache([300, 64, 1000], std=std, d=128, hq=8, hkv=2)
    c.check_attend(c.attend())


def test_attend_with_lists_of_pages():
    rng = np.random.default_rng(3)
    c = Cache([1000, 17, 0, 640, 333], hq=8, hkv=2, d=128, page=16)
    width = 9
    sel = np.full((5, 2, width), -1, np.int32)
    picks = [[None] * 2 for _ in range(5)]
    for b, n in enumerate(c.lens_np):
        held = OP.pages_for(int(n), 16)
        for h in range(2):
            m = min(width, held)
            pick = list(rng.integers(0, held, m)) if m else []  # any order, a page may come twice
            if m and h == 0:
                pick[0] = held - 1  # the last page, not full, in front
            sel[b, h, :m] = pick
            picks[b][h] = pick
    c.check_attend(c.attend(sel=i32(sel)), picks=picks)


def test_attend_with_pages_shared_by_requests():
    # a prompt of 48 tokens in three requests' tables; the rest of each is its own
    c = Cache([200, 100, 48, 75], hq=8, hkv=2, d=64, page=16)
    c.table_np[1:, :3] = c.table_np[0, :3]
    c.table.copy_(i32(c.table_np))
    c.check_attend(c.attend())


def test_attend_leaves_out_bad_pages_and_reports_them():
    c = Cache([64, 64, 64], page=16)
    bad = c.table_np.copy()
    bad[0, 1], bad[1, 0] = c.n_pages, -5
    c.table.copy_(i32(bad))
    out = c.attend(status="RTVLA_ERR_DEVICE_BOUNDS")
    c.check_attend(out, picks=[[[0, 2, 3]], [[1, 2, 3]], [[0, 1, 2, 3]]])
    c.table.copy_(i32(c.table_np))
    c.lens.copy_(i32([-3, 10 ** 9, 64]))
    c.check_attend(c.attend(status="RTVLA_ERR_DEVICE_BOUNDS"), rows=[2])
    assert not c.attend(status="RTVLA_ERR_DEVICE_BOUNDS")[0].any()  # the negative length counts as 0
    c.lens.copy_(c_lens := i32(c.lens_np))
    sel = i32([[[0, 4]], [[-1, 2]], [[2 ** 30, 3]]])
    c.check_attend(c.attend(sel=sel, status="RTVLA_ERR_DEVICE_BOUNDS"), picks=[[[0]], [[2]], [[3]]])
    assert c.attend().isfinite().all() and c_lens is not None


def test_attend_reads_pools_past_32_bit_offsets():
    n_pages, page, d = (1 << 18) + 40, 64, 256
    k = torch.empty((1, n_pages, 1, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 32
    pages = [n_pages - 1, 3, n_pages - 17, 1 << 17]
    for p in pages:
        k[0, p].normal_()
        v[0, p].normal_()
    ctx = R.rtvla_pages_create(R.make_pages_config(n_pages=n_pages, table_width=4, page_size=page, n_layers=1))
    table, lens = i32([pages]), i32([250])
    q = torch.randn((1, 8, d), device="cuda").bfloat16()
    out = torch.empty_like(q)
    R.rtvla_pages_attend(ctx, 0, q, R.make_paged_kv(k, v, None, table, lens, 1), None, 0, out)
    assert R.rtvla_pages_sync_status(ctx) == 0
    kk, vv = (x[0, pages, 0].double().reshape(-1, d)[:250] for x in (k, v))
    w = torch.softmax(q[0].double() @ kk.T / 16, -1)
    ref, size = w @ vv, w @ vv.abs()
    big = float((q[0].double().abs() @ kk.abs().T).max() / 16)
    tol = 2.0 ** -8 * ref.abs() + (2 * 260 * E32 * big + 640 * E32 + 2.0 ** -16) * size
    assert ((out[0].double() - ref).abs() <= tol).all()
    R.rtvla_pages_destroy(ctx)


# ---------------------------------------------------------------------------------------

def run_plan(c, lens, delta, n_rows, in_place=False):
    B = len(lens)
    table, free, nf = i32(c.table_np), i32(c.free_np), i32([c.n_free])
    lens_in, out = i32(lens), i32([0] * B)
    nf_out = nf if in_place else i32([0])
    kv = R.make_paged_kv(None, None, None, table, lens_in if in_place else out, B)
    slots, positions = (torch.full((n_rows + 8,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    start = torch.full((B + 1,), 99, dtype=torch.int32, device="cuda")
    R.rtvla_pages_plan(c.ctx, lens_in, i32(delta), free, nf, kv, nf_out, slots, positions, start, n_rows)
    status = c.status()
    ref = OP.plan(lens, delta, c.table_np, c.free_np, c.n_free, c.page, c.n_pages, n_rows)
    want = {frozenset(): "RTVLA_OK", frozenset(["no_pages"]): "RTVLA_ERR_NO_PAGES"}.get(
        frozenset(ref["err"]), "RTVLA_ERR_DEVICE_BOUNDS")
    assert status == want
    got = (lens_in if in_place else out, table, nf_out, slots[:n_rows], positions[:n_rows], start)
    for name, x in zip(("lens", "table", "n_free", "slots", "positions", "row_start"), got):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(ref[name]).reshape(-1)), name
    assert np.array_equal(free.cpu().numpy()[: ref["n_free"]], ref["free"][: ref["n_free"]])
    assert (slots[n_rows:] == 99).all() and (positions[n_rows:] == 99).all()
    return ref


@pytest.mark.parametrize("batch, page, longest", [(1, 16, 40), (5, 1, 30), (37, 64, 300), (300, 16, 200),
                                                  (1027, 8, 64), (4096, 32, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_over_a_run_of_steps(batch, page, longest, in_place):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, longest, batch)
    c = Cache(lens, d=64, hq=1, page=page, width=OP.pages_for(2 * longest, page) + 1,
              spare=max(3, batch * OP.pages_for(longest, page) // 3))
    for step in range(4):
        delta = rng.integers(-longest, longest // (step + 1) + 1, batch)
        delta[rng.random(batch) < 0.3] = 1
        if step == 2:
            delta = np.full(batch, -10 ** 6)
        rows = int(np.maximum(delta, 0).sum()) + (step * 7) % 13
        ref = run_plan(c, lens, delta, rows, in_place)
        lens, c.table_np, c.free_np, c.n_free = ref["lens"], ref["table"], ref["free"], ref["n_free"]


def test_plan_of_many_rows_and_of_none():
    c = Cache([0, 5, 0], d=64, hq=1, page=16, width=8200, spare=8300)
    run_plan(c, [0, 5, 0], [100001, 3, 17], 131072)
    run_plan(c, [0, 5, 0], [0, 0, 0], 0)
    run_plan(c, [0, 5, 0], [0, -1, 0], 3)


def test_plan_refusals():
    c = Cache([10, 20, 0, 7], d=64, hq=1, page=4, width=8, spare=4)
    run_plan(c, [10, 20, 0, 7], [2, 9, 9, 1], 40)             # the third finds too few pages, the last needs none
    run_plan(c, [10, 20, 0, 7], [-4, 9, 9, 1], 40)            # a page given back is enough for it
    run_plan(c, [10, 20, 0, 7], [2, 13, 3, 1], 40)            # past the table's width
    run_plan(c, [10, 20, 0, 7], [2, 2, 3, 1], 6)              # past the rows
    run_plan(c, [-1, 20, 0, 99], [2, 2, -3, 1], 20)           # lengths that cannot be
    run_plan(c, [10, 20, 0, 7], [2 ** 31 - 1, 2, 2 ** 31 - 1, 1], 16)
    c.n_free = c.n_pages + 9
    run_plan(c, [10, 20, 0, 7], [1, 1, 0, 1], 8)


# ---------------------------------------------------------------------------------------

def rows_for(c, lens, new):
    """Slots and positions of `new[b]` tokens after lens[b], pages taken from the cache's free list."""
    ref = OP.plan(lens, new, c.table_np, c.free_np, c.n_free, c.page, c.n_pages, int(sum(new)))
    assert not ref["err"]
    c.table_np, c.free_np, c.n_free = ref["table"], ref["free"], ref["n_free"]
    return ref["slots"], ref["positions"]


@pytest.mark.parametrize("src", ["same", "f32"])
@pytest.mark.parametrize("dtype, hq, hkv, d, page, theta", [
    ("bf16", 8, 1, 256, 16, 10000.0), ("f16", 8, 2, 128, 64, 500000.0), ("bf16", 3, 3, 64, 1, 10000.0),
    ("f16", 1, 1, 64, 256, 0.0), ("bf16", 32, 4, 128, 32, 0.0), ("bf16", 5, 1, 64, 2, 10000.0)])
def test_write_rows_pools_and_means(dtype, src, hq, hkv, d, page, theta):
    lens, new = [0, 5, 100, 255, 64, 31], [1, 300, 0, 1, 70, 33]
    c = Cache(lens, dtype, hq, hkv, d, page, layers=2, theta=theta, width=OP.pages_for(400, page), spare=700)
    slots, pos = rows_for(c, lens, new)
    # a skipped row between requests and skipped rows at the end
    slots = np.concatenate([slots[:1], [-1], slots[1:], [-1] * 5]).astype(np.int32)
    pos = np.concatenate([pos[:1], [0], pos[1:], [0] * 5]).astype(np.int32)
    T = len(slots)
    qkv = torch.randn((T, (hq + 2 * hkv) * d), device="cuda")
    qkv = qkv if src == "f32" else qkv.to(c.t)
    before = [x.clone() for x in (c.k, c.v, c.k_mean)]
    q_out = torch.full((T, hq, d), 555.0, dtype=c.t, device="cuda")
    code = R.DTYPE_F32 if src == "f32" else c.cfg.dtype
    R.rtvla_pages_write(c.ctx, 1, qkv, code, i32(slots), i32(pos), T, c.kv, q_out)
    assert c.status() == "RTVLA_OK"
    x = qkv.double().cpu().numpy()
    q, k, v = OP.write(x, slots, pos, hq, hkv, theta)
    x = np.abs(x.reshape(T, hq + 2 * hkv, d))
    pair = np.concatenate([x[..., : d // 2] + x[..., d // 2:]] * 2, -1) * 7 * E32
    pair += 2.0 ** -25 if c.f16 else 0.0
    live = slots >= 0
    got_q = q_out.double().cpu().numpy()
    assert (got_q[~live] == float(torch.tensor(555.0).to(c.t))).all()  # the fill as the type holds it
    assert (np.abs(got_q - q) <= c.u * np.abs(q) + pair[:, :hq])[live].all()
    sl = torch.from_numpy(slots[live].astype(np.int64)).cuda()
    v_tol = np.full_like(pair[:, hq:hq + hkv], 2.0 ** -25 if c.f16 else 0.0)
    for pool, old, ref, tol in ((c.k, before[0], k, pair[:, hq:hq + hkv]), (c.v, before[1], v, v_tol)):
        got = pool[1, sl // page, :, sl % page].double().cpu().numpy()
        assert (np.abs(got - ref[live]) <= c.u * np.abs(ref[live]) + tol[live]).all()
        old[1, sl // page, :, sl % page] = pool[1, sl // page, :, sl % page]
        assert torch.equal(pool.view(torch.int16), old.view(torch.int16))  # no other slot, no other layer
    full = sl[sl % page == page - 1] // page
    stored = c.k[1, full].double()
    ref = stored.mean(2)
    tol = c.u * ref.abs() + page * E32 * stored.abs().mean(2) + (2.0 ** -25 if c.f16 else 0.0)
    assert len(full) and ((c.k_mean[1, full].double() - ref).abs() <= tol).all()
    before[2][1, full] = c.k_mean[1, full]
    assert torch.equal(c.k_mean.view(torch.int16), before[2].view(torch.int16))


def test_write_far_positions_and_without_means():
    c = Cache([0], d=128, hq=2, page=1024, width=1 << 14, spare=3)
    far = np.array([(1 << 24) - 1, 8388607, 131071, 65536, 255, 256, 1], np.int32)
    slots = np.arange(7, dtype=np.int32)
    qkv = torch.randn((7, 4 * 128), device="cuda")
    q_out = torch.empty((7, 2, 128), dtype=c.t, device="cuda")
    kv = R.make_paged_kv(c.k, c.v, None, None, None, 0)
    R.rtvla_pages_write(c.ctx, 0, qkv, R.DTYPE_F32, i32(slots), i32(far), 7, kv, q_out)
    assert c.status() == "RTVLA_OK"
    q, k, _ = OP.write(qkv.cpu().numpy(), slots, far, 2, 1, 10000.0)
    x = np.abs(qkv.double().cpu().numpy().reshape(7, 4, 128))
    # the oracle's own fp64 angle at 2^24 is off by 2^24 * 2^-53
    tol = np.concatenate([x[..., :64] + x[..., 64:]] * 2, -1) * 8 * E32
    assert (np.abs(q_out.double().cpu().numpy() - q) <= c.u * np.abs(q) + tol[:, :2]).all()
    assert (np.abs(c.k[0, 0, 0, :7].double().cpu().numpy() - k[:, 0]) <= c.u * np.abs(k[:, 0]) + tol[:, 2]).all()
    R.rtvla_pages_write(c.ctx, 0, None, R.DTYPE_F32, None, None, 0, kv, None)  # no rows


def test_write_skips_bad_slots_and_positions():
    c = Cache([16], d=64, hq=1, page=16, width=2)
    before = [x.clone() for x in (c.k, c.v, c.k_mean)]
    cap = c.n_pages * 16
    slots = i32([-2, cap, 2 ** 31 - 1, -2 ** 31, 0, 1])
    pos = i32([0, 0, 0, 0, -1, 32])
    q_out = torch.full((6, 64), 5.0, dtype=c.t, device="cuda")
    R.rtvla_pages_write(c.ctx, 0, torch.randn((6, 192), device="cuda"), R.DTYPE_F32, slots, pos, 6, c.kv, q_out)
    assert c.status() == "RTVLA_ERR_DEVICE_BOUNDS"
    assert (q_out == 5.0).all()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(before, (c.k, c.v, c.k_mean)))


# ---------------------------------------------------------------------------------------

def check_select(c, sel, budget, first, last, layer=0):
    q, means, got = c.q.double().cpu().numpy(), c.k_mean[layer].double().cpu().numpy(), sel.cpu().numpy()
    G = c.hq // c.hkv
    for b, n in enumerate(c.lens_np):
        held = OP.pages_for(int(n), c.page)
        for h in range(c.hkv):
            s = OP.scores(q[b, h * G:(h + 1) * G], means[c.table_np[b, :held], h])
            ref = OP.choose(s, held, budget, first, last)
            assert list(got[b, h]) == ref + [-1] * (budget - len(ref)), (b, h, held)


@pytest.mark.parametrize("dtype, hq, hkv, d, page, budget, first, last", [
    ("bf16", 8, 1, 256, 16, 16, 1, 2), ("f16", 8, 4, 64, 8, 7, 0, 1), ("bf16", 16, 1, 128, 1, 100, 3, 5),
    ("f16", 3, 3, 128, 4, 9, 4, 5), ("bf16", 4, 2, 64, 2, 1, 0, 1), ("bf16", 8, 1, 256, 16, 300, 1, 1)])
def test_select_matches_the_oracle(dtype, hq, hkv, d, page, budget, first, last):
    c = Cache([3000, 0, 1, page * budget, page * budget + 1, 2049, 777], dtype, hq, hkv, d, page, layers=2)
    sel = torch.full((7, hkv, budget), 5, dtype=torch.int32, device="cuda")
    R.rtvla_pages_select(c.ctx, 1, c.q, c.kv, budget, first, last, sel)
    assert c.status() == "RTVLA_OK"
    check_select(c, sel, budget, first, last, 1)


def test_select_with_equal_scores_and_extreme_ones():
    c = Cache([16 * 500, 16 * 500, 16 * 500, 16 * 4000], page=16, d=64, hq=2)
    m = c.k_mean[0]
    m[c.table[0, :500].long()] = 1.0                       # all equal: the lowest pages
    m[c.table[1, :500].long()] = m[c.table[1, 5]].clone()  # two values only
    m[c.table[1, 100:400:3].long()] *= 2
    m[c.table[2, :500].long()] *= torch.logspace(-4, 4, 500, device="cuda")[:, None, None].bfloat16()
    c.q[1] = 0.0                                           # every score 0
    for budget in (3, 64, 257):
        sel = torch.empty((4, 1, budget), dtype=torch.int32, device="cuda")
        R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, budget, 1, 1, sel)
        assert c.status() == "RTVLA_OK"
        check_select(c, sel, budget, 1, 1)
    c.q[1] = 1.0
    sel = torch.empty((4, 1, 90), dtype=torch.int32, device="cuda")
    R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, 90, 0, 1, sel)
    assert c.status() == "RTVLA_OK"
    check_select(c, sel, 90, 0, 1)


@pytest.mark.parametrize("page, tokens", [(1, 20000), (2, 70001)])
def test_select_over_tables_longer_than_shared_memory(page, tokens):
    c = Cache([tokens, 300, tokens - 77], d=64, hq=4, hkv=2, page=page)
    m = c.k_mean[0]
    m[c.table[2, 100:15000].long()] = 0.5  # thousands of equal scores around the cut
    for budget in (100, 5000):
        sel = torch.empty((3, 2, budget), dtype=torch.int32, device="cuda")
        R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, budget, 2, 3, sel)
        assert c.status() == "RTVLA_OK"
        check_select(c, sel, budget, 2, 3)


def test_select_with_scores_closer_than_fp32_can_tell():
    """Pages whose scores differ by less than an fp32 sum's rounding, and infinite ones."""
    c = Cache([16 * 900, 16 * 900], page=16, d=128, hq=1)
    rng = np.random.default_rng(11)
    base = rng.normal(size=128).astype(np.float32) * 64
    pages = c.table[0, :900].long()
    m = torch.from_numpy(np.tile(base, (900, 1))).cuda().bfloat16()
    m[:, 0] = torch.from_numpy(rng.integers(-3, 4, 900).astype(np.float32) * 2.0 ** -30).cuda().bfloat16()
    c.k_mean[0, pages, 0] = m
    pages = c.table[1, :900].long()
    c.k_mean[0, pages[5:50:7], 0, 3] = float("inf")
    c.k_mean[0, pages[6:800:7], 0, 3] = float("-inf")
    c.q[1] = c.q[1].abs() + 0.125
    for budget in (40, 400, 880):
        sel = torch.empty((2, 1, budget), dtype=torch.int32, device="cuda")
        R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, budget, 0, 2, sel)
        assert c.status() == "RTVLA_OK"
        check_select(c, sel, budget, 0, 2)


def test_select_puts_bad_pages_last_and_reports_them():
    c = Cache([16 * 40], d=64, hq=1, page=16)
    bad = c.table_np.copy()
    bad[0, [3, 17]] = [-1, c.n_pages]
    c.table.copy_(i32(bad))
    sel = torch.empty((1, 1, 38), dtype=torch.int32, device="cuda")
    R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, 38, 0, 1, sel)
    assert c.status() == "RTVLA_ERR_DEVICE_BOUNDS"
    assert list(sel.cpu().numpy()[0, 0]) == [e for e in range(40) if e not in (3, 17)]


# ---------------------------------------------------------------------------------------

def test_steps_together_as_a_captured_graph():
    """Decode steps of a ragged batch over two layers: plan in place, then per layer write, select and
    attend; captured once, replayed, every step checked against the oracle on the pool as it stands."""
    lens = [37, 0, 250, 16]
    c = Cache(lens, hq=8, hkv=2, d=64, page=16, layers=2, width=30, spare=40)
    B, T, budget = 4, 6, 6
    delta, free, nf = i32([1, 1, 1, 1]), i32(c.free_np), i32([c.n_free])
    slots, pos, start = i32([0] * T), i32([0] * T), i32([0] * (B + 1))
    qkv = torch.zeros((2, T, 12 * 64), dtype=c.t, device="cuda")
    q = torch.zeros((T, 8, 64), dtype=c.t, device="cuda")
    qs, sel = [torch.zeros_like(c.q) for _ in range(2)], [i32(np.zeros((B, 2, budget))) for _ in range(2)]
    out, full = ([torch.zeros_like(c.q) for _ in range(2)] for _ in range(2))

    def step(stream):
        R.rtvla_pages_plan(c.ctx, c.lens, delta, free, nf, c.kv, nf, slots, pos, start, T, stream)
        for l in range(2):
            R.rtvla_pages_write(c.ctx, l, qkv[l], c.cfg.dtype, slots, pos, T, c.kv, q, stream)
            qs[l].copy_(q[:B])
            R.rtvla_pages_select(c.ctx, l, q, c.kv, budget, 1, 1, sel[l], stream)
            R.rtvla_pages_attend(c.ctx, l, q, c.kv, sel[l], budget, out[l], stream)
            R.rtvla_pages_attend(c.ctx, l, q, c.kv, None, 0, full[l], stream)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for i in range(20):
        if i == 7:
            delta.copy_(i32([1, 1, -13, 1]))  # the third request drops the end of a full page, then refills it
        if i == 8:
            delta.copy_(i32([1, 1, 1, 1]))
        qkv.normal_()
        d = delta.cpu().numpy()
        ref = OP.plan(c.lens_np, d, c.table_np, c.free_np, c.n_free, 16, c.n_pages, T)
        graph.replay()
        assert c.status() == "RTVLA_OK"
        c.lens_np, c.table_np, c.free_np, c.n_free = ref["lens"], ref["table"], ref["free"], ref["n_free"]
        assert np.array_equal(slots.cpu().numpy(), ref["slots"]) and int(nf) == ref["n_free"]
        assert np.array_equal(c.lens.cpu().numpy(), ref["lens"])
        for l in range(2):
            c.q = qs[l]
            check_select(c, sel[l], budget, 1, 1, l)
            picks = [[[e for e in row if e >= 0] for row in req] for req in sel[l].cpu().numpy()]
            c.check_attend(out[l], l, picks)
            c.check_attend(full[l], l)
    # every full page's mean is that of the keys it holds now, pages filled a second time among them
    for b, n in enumerate(c.lens_np):
        pages = c.table_np[b, : n // 16].astype(np.int64)
        for l in range(2):
            keys = c.k[l, pages].double().cpu().numpy()
            ref, got = keys.mean(2), c.k_mean[l, pages].double().cpu().numpy()
            assert (np.abs(got - ref) <= c.u * np.abs(ref) + 16 * E32 * np.abs(keys).mean(2)).all()


def test_contexts_on_two_streams_at_once():
    cs = [Cache([700 + 100 * i, 3000, 5], seed=i + 1, d=128, hq=8) for i in range(2)]
    outs = [torch.zeros_like(c.q) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, o, s in zip(cs, outs, streams):
            R.rtvla_pages_attend(c.ctx, 0, c.q, c.kv, None, 0, o, s)
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check_attend(o)


def test_repeated_calls_give_equal_bits():
    c = Cache([5000, 17, 900, 64], hq=8, d=256)
    first = c.attend()
    for _ in range(10):
        assert torch.equal(first, c.attend())


def test_guard_bands_hold(monkeypatch):
    monkeypatch.setenv("RTVLA_CHECKED", "1")
    c = Cache([5000, 0, 17], hq=16, hkv=1, d=256, page=16)
    c.check_attend(c.attend())
    sel = i32(np.zeros((3, 1, 20)))
    R.rtvla_pages_select(c.ctx, 0, c.q, c.kv, 20, 1, 1, sel)
    assert c.status() == "RTVLA_OK"
    check_select(c, sel, 20, 1, 1)
    run_plan(c, [5000, 0, 17], [3, 40, -17], 50)


def test_a_capped_context_is_refused(monkeypatch):
    monkeypatch.setenv("RTVLA_DEVICE_MEMORY_CAP", "4096")
    with pytest.raises(R.RtvlaError) as e:
        R.rtvla_pages_create(R.make_pages_config(n_pages=4, table_width=4))
    assert e.value.name == "RTVLA_ERR_OOM"


def test_argument_errors():
    c = Cache([40, 3], hq=2, d=64)
    out, sel = torch.empty_like(c.q), i32(np.zeros((2, 1, 2)))
    slots, qkv = i32([0, 1]), torch.zeros((2, 256), device="cuda")

    def fails(name, fn, *args):
        with pytest.raises(R.RtvlaError) as e:
            fn(c.ctx, *args)
        assert e.value.name == "RTVLA_ERR_" + name

    big = R.make_paged_kv(c.k, c.v, c.k_mean, c.table, c.lens, 3)
    none = R.make_paged_kv(c.k, None, c.k_mean, c.table, c.lens, 2)
    odd = R.make_paged_kv(c.k.data_ptr() + 2, c.v, c.k_mean, c.table, c.lens, 2)
    blind = R.make_paged_kv(c.k, c.v, None, c.table, c.lens, 2)
    at, se, wr, pl = R.rtvla_pages_attend, R.rtvla_pages_select, R.rtvla_pages_write, R.rtvla_pages_plan
    fails("SHAPE", at, 0, c.q, big, None, 0, out)
    fails("SHAPE", at, 1, c.q, c.kv, None, 0, out)
    fails("INVALID_ARG", at, -1, c.q, c.kv, None, 0, out)
    fails("INVALID_ARG", at, 0, c.q, none, None, 0, out)
    fails("INVALID_ARG", at, 0, c.q, odd, None, 0, out)
    fails("INVALID_ARG", at, 0, c.q.data_ptr() + 2, c.kv, None, 0, out)
    fails("INVALID_ARG", at, 0, c.q, c.kv, None, 0, None)
    fails("INVALID_ARG", at, 0, c.q, c.kv, sel, 0, out)
    fails("SHAPE", at, 0, c.q, c.kv, sel, 65537, out)
    fails("INVALID_ARG", se, 0, c.q, blind, 2, 0, 1, sel)
    fails("INVALID_ARG", se, 0, c.q, c.kv, 2, 0, 0, sel)
    fails("INVALID_ARG", se, 0, c.q, c.kv, 2, 2, 1, sel)
    fails("INVALID_ARG", se, 0, c.q, c.kv, 2, -1, 1, sel)
    fails("SHAPE", se, 0, c.q, c.kv, 65537, 0, 1, sel)
    fails("INVALID_ARG", wr, 0, qkv, R.DTYPE_F16, slots, slots, 2, c.kv, out)
    fails("INVALID_ARG", wr, 0, qkv, R.DTYPE_F32, slots, slots, -1, c.kv, out)
    fails("INVALID_ARG", wr, 0, qkv, R.DTYPE_F32, None, slots, 2, c.kv, out)
    fails("INVALID_ARG", wr, 0, qkv.data_ptr() + 4, R.DTYPE_F32, slots, slots, 2, c.kv, out)
    fails("SHAPE", wr, 1, qkv, R.DTYPE_F32, slots, slots, 2, c.kv, out)
    fails("SHAPE", wr, 0, qkv, R.DTYPE_F32, slots, slots, (1 << 24) + 1, c.kv, out)
    free, nf = i32(c.free_np), i32([c.n_free])
    fails("INVALID_ARG", pl, c.lens, c.lens, free, nf, c.kv, nf, None, slots, slots, 2)
    fails("INVALID_ARG", pl, c.lens, c.lens, free, nf, c.kv, nf, slots, slots, None, 2)
    fails("SHAPE", pl, c.lens, c.lens, free, nf, big, nf, slots, slots, slots, 2)
    fails("SHAPE", pl, c.lens, c.lens, free, nf, c.kv, nf, slots, slots, slots, (1 << 24) + 1)
    lean = R.rtvla_pages_create(R.make_pages_config(n_pages=c.n_pages, table_width=c.width, n_layers=1, n_q_heads=2,
                                                    head_dim=64, max_batch=2, has_select=False))
    with pytest.raises(R.RtvlaError) as e:
        se(lean, 0, c.q, c.kv, 2, 0, 1, sel)
    assert e.value.name == "RTVLA_ERR_UNSUPPORTED"
    R.rtvla_pages_destroy(lean)
    assert c.status() == "RTVLA_OK"
