"""rtvla_prefix_step at batches on both sides of the GEMMs' token tiles (64, 128, 256), and with a request
that a plan refused, against the fp64 oracle.  Tolerances: the prefix pass's own (tests/harness.py)."""
import numpy as np
import pytest
import torch

import flow_matching_action_expert_b200 as R
from oracle import pages as OP
from synth import gen
from synth import workloads as WL

from harness import H_REL_L2, KV_REL_L2, GpuModel, bf16_dev, rel_l2

pytestmark = pytest.mark.gpu

PAGE, WIDTH, MAX = 16, 4, 129


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def model():
    base = WL.workload(1)
    wl = WL.Workload("step L2 B129", base.expert, base.chunk, MAX, 32, (32,) * MAX,
                     prefill=WL.PrefillShape(n_layers=base.expert.n_layers))
    pbits = WL.prefill_weights(wl.prefill)
    m = GpuModel(wl, WL.expert_weights(wl.expert, stressed=True), prefill_bits=pbits)
    yield wl, m, {k: v.astype(np.float64) for k, v in WL.as_f32(pbits).items()}
    m.close()


@pytest.mark.parametrize("batch, refused", [(1, ()), (64, (63,)), (65, (0,)), (128, ()), (129, (64, 127))])
def test_step_of_a_batch(model, batch, refused):
    wl, m, W = model
    L, rng = wl.prefill.n_layers, np.random.default_rng(batch)
    lens = rng.integers(0, WIDTH * PAGE, batch)  # tokens before the step
    n_pages = batch * WIDTH + 2
    table = rng.permutation(n_pages)[:batch * WIDTH].reshape(batch, WIDTH)
    pool = [bf16_dev(gen.normal_bf16(f"batches/{batch}/{n}", (L, n_pages, 1, PAGE, 256), 1.0)) for n in "kv"]
    before = [x.clone() for x in pool]
    after, slots = lens + 1, table[np.arange(batch), lens // PAGE] * PAGE + lens % PAGE
    for b in refused:
        after[b], slots[b] = lens[b], -1
    pages = R.rtvla_pages_create(R.make_pages_config(n_pages=n_pages, table_width=WIDTH, page_size=PAGE, n_layers=L,
                                                     max_batch=batch, has_select=False))
    tab, held_now = i32(table), i32(after)
    kv = R.make_paged_kv(*pool, None, tab, held_now, batch)
    e = gen.normal_bf16(f"batches/{batch}/embeds", (batch, 2048), np.sqrt(2048))
    hidden = torch.zeros((batch, 2048), dtype=torch.float32, device="cuda")
    pos = np.where(slots < 0, 0, lens)
    R.rtvla_prefix_step(m.ctx, pages, bf16_dev(e), i32(slots), i32(pos), kv, hidden)
    assert R.rtvla_pages_sync_status(pages) == 0 and R.rtvla_sync_status(m.ctx) == 0
    live = slots[slots >= 0]
    for x, old in zip(pool, before):  # nothing but the new rows
        old[:, live // PAGE, 0, live % PAGE] = x[:, live // PAGE, 0, live % PAGE]
        assert torch.equal(x.view(torch.int16), old.view(torch.int16))
    K, V = (x.double().cpu().numpy() for x in pool)
    got, e = hidden.double().cpu().numpy(), gen.bf16_to_f32(e)
    for b in sorted({0, 1, 62, 63, 64, 126, 127, 128} & set(range(batch)) - set(refused)):
        held = [[OP.keys_of(x[l], table[b], int(lens[b]), 0, PAGE) for l in range(L)] for x in (K, V)]
        x, k, v = OP.prefix_step(W, wl.prefill, e[b], *held, int(lens[b]))
        assert rel_l2(got[b], x) <= H_REL_L2 and rel_l2(got[b] - e[b], x - e[b]) <= H_REL_L2, b
        for l in range(L):
            s = slots[b]
            assert rel_l2(K[l, s // PAGE, 0, s % PAGE], k[l]) <= KV_REL_L2
            assert rel_l2(V[l, s // PAGE, 0, s % PAGE], v[l]) <= KV_REL_L2
    R.rtvla_pages_destroy(pages)
