"""The prefix model's step for one new token per request on a paged cache (rtvla_prefix_step),
after rtvla_prefill, against the fp64 oracle, and on into the denoise loop.

Tolerances are the prefix pass's own (tests/harness.py): relative L2 1e-2 of the cache's rows and of
the hidden state's update, 3e-2 / 1e-2 of the actions.  The oracle starts from the GPU's prefilled
cache, so that only the steps are compared.
"""
import numpy as np
import pytest
import torch

import flow_matching_action_expert_b200 as R
from oracle import model as O
from oracle import pages as OP
from synth import gen
from synth import workloads as WL

from harness import H_REL_L2, KV_REL_L2, GpuModel, assert_actions_close, bf16_dev, rel_l2

pytestmark = pytest.mark.gpu

PAGE, CAP, LENS = 16, 288, (200, 17, 64)
STEPS = 4


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def model():
    base = WL.workload(1)
    wl = WL.Workload("step L2 P288 B3", base.expert, base.chunk, 3, CAP, LENS,
                     prefill=WL.PrefillShape(n_layers=base.expert.n_layers))
    ebits, pbits = WL.expert_weights(wl.expert, stressed=True), WL.prefill_weights(wl.prefill)
    m = GpuModel(wl, ebits, prefill_bits=pbits)
    emb, mask = WL.prefill_inputs(wl)
    new = gen.normal_bf16("step/embeds", (STEPS, 3, 2048), np.sqrt(2048))
    yield wl, m, WL.as_f32(ebits), WL.as_f32(pbits), emb, mask, new
    m.close()


def host(t):
    return t.double().cpu().numpy()


def check(wl, W, embed, hidden, k_new, v_new, K, V, pos):
    x, k, v = OP.prefix_step(W, wl.prefill, embed, K, V, pos)
    assert rel_l2(hidden, x) <= H_REL_L2
    assert rel_l2(hidden - embed, x - embed) <= H_REL_L2
    for l in range(wl.prefill.n_layers):
        assert rel_l2(k_new[l], k[l]) <= KV_REL_L2 and rel_l2(v_new[l], v[l]) <= KV_REL_L2


def test_steps_on_scattered_pages_captured_and_direct(model):
    wl, m, _, W, emb, mask, new = model
    L, B, width = 2, 3, 20
    k, v, valid = m.prefill(emb, mask)
    n_pages = B * CAP // PAGE + 9
    order = np.random.default_rng(2).permutation(n_pages)
    pool_k = torch.full((L, n_pages, 1, PAGE, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool_v = pool_k.clone()
    table, at = np.full((B, width), -1, np.int32), 0
    for b, n in enumerate(LENS):
        for i in range(OP.pages_for(n, PAGE)):
            table[b, i] = p = order[at]
            at += 1
            pool_k[:, p, 0], pool_v[:, p, 0] = k[:, b, i * PAGE:][:, :PAGE], v[:, b, i * PAGE:][:, :PAGE]
    free = i32(np.concatenate([order[at:], np.zeros(at)]))
    nf, lens, tab = i32([n_pages - at]), i32(LENS), i32(table)
    pages = R.rtvla_pages_create(R.make_pages_config(n_pages=n_pages, table_width=width, page_size=PAGE, n_layers=L,
                                                     max_batch=B, has_select=False))
    kv = R.make_paged_kv(pool_k, pool_v, None, tab, lens, B)
    one, slots, pos, start = i32([1] * B), i32([0] * B), i32([0] * B), i32([0] * (B + 1))
    x = torch.zeros((B, 2048), dtype=torch.bfloat16, device="cuda")
    hidden = torch.zeros((B, 2048), dtype=torch.float32, device="cuda")

    def step(stream=None):
        R.rtvla_pages_plan(pages, lens, one, free, nf, kv, nf, slots, pos, start, B, stream)
        R.rtvla_prefix_step(m.ctx, pages, x, slots, pos, kv, hidden, stream)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    held = [[list(host(t[l, b, :n])) for b, n in enumerate(LENS)] for t in (k, v) for l in range(L)]
    for s in range(STEPS):
        x.copy_(bf16_dev(new[s]))
        graph.replay() if s % 2 else step()
        assert R.rtvla_pages_sync_status(pages) == 0 and R.rtvla_sync_status(m.ctx) == 0
        sl, hid, e = slots.cpu().numpy(), host(hidden), gen.bf16_to_f32(new[s])
        assert list(pos.cpu().numpy()) == [n + s for n in LENS]
        for b in range(B):
            kn, vn = (host(t[:, sl[b] // PAGE, 0, sl[b] % PAGE]) for t in (pool_k, pool_v))
            K, V = ([np.array(held[i * L + l][b]) for l in range(L)] for i in range(2))
            check(wl, W, e[b], hid[b], kn, vn, K, V, LENS[b] + s)
            for l in range(L):
                held[l][b].append(kn[l])
                held[L + l][b].append(vn[l])
    R.rtvla_pages_destroy(pages)


def test_steps_on_a_contiguous_cache_then_the_denoise_loop(model):
    """The prefix cache of rtvla_prefill seen as a pool: steps extend it, the action expert attends
    to the extended prefix."""
    wl, m, We, W, emb, mask, new = model
    k, v, valid = m.prefill(emb, mask)
    B, width = 3, CAP // PAGE
    pages = R.rtvla_pages_create(R.make_pages_config(n_pages=B * width, table_width=width, page_size=PAGE, n_layers=2,
                                                     max_batch=B, has_select=False))
    tab = i32(np.arange(B * width).reshape(B, width))
    lens = valid.clone()
    kv = R.make_paged_kv(k, v, None, tab, lens, B)
    first = torch.arange(B, device="cuda", dtype=torch.int32) * CAP
    hidden = torch.zeros((B, 2048), dtype=torch.float32, device="cuda")
    for s in range(STEPS):
        slots, pos = first + lens, lens.clone()
        lens += 1
        R.rtvla_prefix_step(m.ctx, pages, bf16_dev(new[s]), slots, pos, kv, hidden)
    assert R.rtvla_pages_sync_status(pages) == 0 and R.rtvla_sync_status(m.ctx) == 0
    Kn, Vn = host(k), host(v)
    noise = WL.noise(wl)
    out = m.sample(noise, k, v, lens)
    full = np.array([n + STEPS for n in LENS], np.int32)
    assert_actions_close(out, O.sample_actions(We, wl.expert, noise, Kn, Vn, full), "after steps")
    # the last step from what the cache held before it
    e = gen.bf16_to_f32(new[STEPS - 1])
    for b in range(B):
        n = LENS[b] + STEPS - 1
        check(wl, W, e[b], host(hidden)[b], Kn[:, b, n], Vn[:, b, n], Kn[:, b, :n], Vn[:, b, :n], n)
    R.rtvla_pages_destroy(pages)


def test_step_refuses_a_cache_that_is_not_the_models(model):
    wl, m, _, _, _, _, _ = model
    t = i32([[0]])
    x = torch.zeros((4, 2048), dtype=torch.float32, device="cuda")

    def refused(name, batch=1, **kw):
        args = dict(n_pages=4, table_width=1, page_size=PAGE, n_layers=2, max_batch=4, has_select=False)
        args.update(kw)
        pages = R.rtvla_pages_create(R.make_pages_config(**args))
        kv = R.make_paged_kv(x, x, None, t, t, batch)
        with pytest.raises(R.RtvlaError) as e:
            R.rtvla_prefix_step(m.ctx, pages, x, t, t, kv, x)
        assert e.value.name == "RTVLA_ERR_" + name
        R.rtvla_pages_destroy(pages)

    refused("UNSUPPORTED", n_layers=3)
    refused("UNSUPPORTED", head_dim=128)
    refused("UNSUPPORTED", dtype=R.DTYPE_F16)
    refused("UNSUPPORTED", rope_theta=500000.0)
    refused("UNSUPPORTED", n_q_heads=16)
    refused("SHAPE", batch=4)
    refused("SHAPE", batch=3, max_batch=2)
    refused("INVALID_ARG", batch=0)
