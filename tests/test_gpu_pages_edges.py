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
from test_gpu_pages import Cache, check_select

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
