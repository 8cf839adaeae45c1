"""The paged KV cache's operators, as measured: cases, plain forms, and the calls a user makes.

Four operators of the paged cache (include/rtvla.h, rtvla_pages_*):

  plan    block tables, slots and positions of a step's new tokens, from request lengths
  write   RoPE on Q and K, K and V into their slots, the mean key of every page that fills up
  attend  attention of one new token per request over its pages
  sparse  the same over the pages a score (summed query . mean key) selects for each KV head

With `own` false `run` computes them in elementary torch operations; with `own` true it calls the
library.  Request lengths come from the case alone, every tensor's contents from the seed.
"""
from __future__ import annotations

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
THETA = 10000.0


def listed():
    """The cases, smallest to largest within an operator."""
    return [
        # one robot decoding text after a 2-view prefix (512 image tokens and a short prompt)
        dict(name="attend-one-robot", op="attend", dtype="bf16", batch=1, q_heads=8, kv_heads=1, head_dim=256,
             page=16, min_len=544, max_len=544, spread=1),
        # a fleet of 16 robots on 3 views, prompts of different length
        dict(name="attend-fleet", op="attend", dtype="bf16", batch=16, q_heads=8, kv_heads=1, head_dim=256,
             page=16, min_len=768, max_len=816, spread=2),
        # one robot with a long history of frames; an odd length that ends inside a page
        dict(name="attend-long-history", op="attend", dtype="bf16", batch=1, q_heads=8, kv_heads=1, head_dim=256,
             page=64, min_len=131071, max_len=131071, spread=3),
        # grouped heads of width 128 in half precision, very ragged lengths from one token on
        dict(name="attend-grouped-f16", op="attend", dtype="f16", batch=24, q_heads=32, kv_heads=8, head_dim=128,
             page=16, min_len=1, max_len=8192, spread=4),
        # the largest: 64 robots with histories up to 32768 tokens
        dict(name="attend-fleet-history", op="attend", dtype="bf16", batch=64, q_heads=8, kv_heads=1, head_dim=256,
             page=64, min_len=512, max_len=32768, spread=5),
        # narrow heads, a few requests, a small budget of pages with the prompt's page kept
        dict(name="sparse-narrow-f16", op="sparse", dtype="f16", batch=4, q_heads=16, kv_heads=4, head_dim=64,
             page=16, min_len=1500, max_len=3001, spread=6, budget=32, keep_first=1, keep_last=2),
        # one robot with a long history that attends to 64 of its 2048 pages
        dict(name="sparse-long-history", op="sparse", dtype="bf16", batch=1, q_heads=8, kv_heads=1, head_dim=256,
             page=64, min_len=131071, max_len=131071, spread=7, budget=64, keep_first=4, keep_last=4),
        # a fleet with histories: every request attends to at most 128 pages
        dict(name="sparse-fleet", op="sparse", dtype="bf16", batch=32, q_heads=8, kv_heads=1, head_dim=256,
             page=32, min_len=1024, max_len=65536, spread=8, budget=128, keep_first=8, keep_last=4),
        # one decode step of 64 requests: one new token each
        dict(name="plan-decode", op="plan", batch=64, page=16, max_len=816, spread=9, new=1, release=0.0, pad=0),
        # a step that admits prompts, decodes, rolls back and releases, rows padded to a fixed count
        dict(name="plan-mixed", op="plan", batch=2000, page=16, max_len=4096, spread=10, new=256, release=0.2,
             pad=1000),
        # the decode step's write, from the QKV product's fp32 sums
        dict(name="write-decode", op="write", dtype="bf16", qkv="f32", batch=16, q_heads=8, kv_heads=1, head_dim=256,
             page=16, max_len=816, spread=11, new=1, pad=0),
        # 16 prompts of up to 544 tokens written at once, after what the requests already hold
        dict(name="write-prompts", op="write", dtype="bf16", qkv="bf16", batch=16, q_heads=8, kv_heads=1,
             head_dim=256, page=32, max_len=300, spread=12, new=544, pad=13),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(("attend", "sparse", "plan", "write"))
    spread = rng.randrange(1, 1 << 30)
    page = rng.choice((1, 8, 16, 32, 64, 128, 256))
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 2000), page=page, max_len=_log(rng, 16, 4096), spread=spread,
                    new=_log(rng, 1, 256), release=rng.choice((0.0, 0.1, 0.3)), pad=rng.choice((0, 1, 37, 500)))
    head_dim = rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 1, 2, 4, 8)) if head_dim < 256 else rng.choice((1, 1, 2))
    q_heads = kv_heads * rng.choice((1, 3, 4, 7, 8, 8, 16))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    case = dict(op=op, dtype=dtype, batch=0, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                spread=spread)
    if op == "write":
        case.update(qkv=rng.choice((dtype, "f32")), batch=_log(rng, 1, 64), max_len=_log(rng, 16, 2000),
                    new=rng.choice((1, _log(rng, 1, 300))), pad=rng.choice((0, 5, 64)))
        case["batch"] = max(1, min(case["batch"], 300000 // (case["new"] * (q_heads + 2 * kv_heads))))
        return case
    # at most about a third of the largest listed case's keys x KV width
    case["batch"] = _log(rng, 1, 64)
    longest = max(64, min(131072, (170 << 20) // (case["batch"] * kv_heads * head_dim)))
    case["max_len"] = _log(rng, 64, longest)
    case["min_len"] = rng.choice((1, case["max_len"], 1 + case["max_len"] // 2))
    if op == "sparse":
        case["page"] = rng.choice((8, 16, 32, 64, 128, 256))
        case["keep_first"] = rng.choice((0, 1, 4))
        case["keep_last"] = rng.choice((1, 2, 4))
        case["budget"] = rng.choice((8, 17, 32, 64, 100, 128))
    return case


# ---------------------------------------------------------------------------------------
# request lengths and what follows from them (the case alone decides these)

def _pages(n, page):
    return -(-n // page)


def _lens(case):
    r = random.Random(case["spread"])
    if case["op"] in ("attend", "sparse"):
        lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"])]
        lens[r.randrange(len(lens))] = case["max_len"]
        return lens, None
    lens = [r.randint(0, case["max_len"]) for _ in range(case["batch"])]
    delta = []
    for n in lens:
        u = r.random()
        if u < case.get("release", 0.0):  # half of these roll a few tokens back, half release all
            delta.append(-r.randint(1, 8) if r.random() < 0.5 else -n)
        else:
            delta.append(case["new"] if case["new"] == 1 else r.randint(0, case["new"]))
    delta[-1] = max(1, delta[-1])
    return lens, delta


def _width(case, lens, delta):
    most = max(max(n, n + d) for n, d in zip(lens, delta or [0] * len(lens)))
    return _pages(most, case["page"]) + 1


def work(case):
    lens, delta = _lens(case)
    page = case["page"]
    if case["op"] == "plan":
        rows = sum(max(d, 0) for d in delta) + case["pad"]
        moved = sum(abs(_pages(max(n + d, 0), page) - _pages(n, page)) for n, d in zip(lens, delta))
        return {"bytes": 4 * (4 * len(lens) + 2 * moved + 2 * rows), "flops": 0}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "write":
        rows = sum(delta)
        filled = sum((n + m) // page - n // page for n, m in zip(lens, delta))
        size = 4 if case["qkv"] == "f32" else 2
        return {"bytes": rows * ((hq + 2 * hkv) * d * (size + 2) + 8) + filled * hkv * d * 2,
                "flops": rows * (hq + hkv) * d * 3}
    keys, means = sum(lens), 0
    if case["op"] == "sparse":
        keys = 0
        for n in lens:
            held = _pages(n, page)
            if held > case["budget"]:
                means += held
                keys += (case["budget"] - 1) * page + n - (held - 1) * page
            else:
                keys += n
    return {"bytes": 4 * keys * hkv * d + 2 * means * hkv * d + 4 * len(lens) * hq * d,
            "flops": 4 * keys * hq * d + 2 * means * hkv * d}


# ---------------------------------------------------------------------------------------
# inputs

class _Pages:
    """The library's handle of one paged cache; destroyed with the state that holds it."""

    def __init__(self, case, n_pages, width):
        import flow_matching_action_expert_b200 as R
        self.R = R
        dtype = R.DTYPE_F16 if case.get("dtype") == "f16" else R.DTYPE_BF16
        cfg = R.make_pages_config(dtype=dtype, n_layers=1, n_q_heads=case.get("q_heads", 8),
                                  n_kv_heads=case.get("kv_heads", 1), head_dim=case.get("head_dim", 256),
                                  page_size=case["page"], n_pages=n_pages, table_width=width,
                                  max_batch=case["batch"], rope_theta=THETA)
        self.ctx = R.rtvla_pages_create(cfg)

    def __del__(self):
        self.R.rtvla_pages_destroy(self.ctx)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _add_handle(st, case)
    return st


def _add_handle(st, case):
    """The handle, the cache's description and the output buffers a user's program keeps."""
    h = st["pages"] = _Pages(case, st["n_pages"], st["table"].shape[1])
    B, lens = case["batch"], st["lens"]

    def empty(*shape):
        return torch.empty(shape, dtype=torch.int32, device="cuda")
    if case["op"] == "plan":
        st.update(lens_out=empty(B), n_free_out=empty(1), slots=empty(st["rows"]), positions=empty(st["rows"]),
                  row_start=empty(B + 1))
        lens = st["lens_out"]
    elif case["op"] != "write":
        st["out"] = torch.empty_like(st["q"])
    if case["op"] == "sparse":
        st["sel"] = empty(B, case["kv_heads"], case["budget"])
    st["kv"] = h.R.make_paged_kv(st.get("k"), st.get("v"), st.get("k_mean"), st["table"], lens, B)


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + case["spread"] % 7919)
    page, B = case["page"], case["batch"]
    lens, delta = _lens(case)
    width = _width(case, lens, delta)
    held = [_pages(n, page) for n in lens]
    after = [_pages(max(n + d, 0), page) for n, d in zip(lens, delta)] if delta else held
    # what the pool holds, and a free list with a few pages to spare
    grow = sum(max(0, a - h) for a, h in zip(after, held))
    back = sum(max(0, h - a) for a, h in zip(after, held))
    spare = max(1, grow - back // 2)
    n_pages = sum(held) + spare + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    hold = torch.tensor(held, device="cuda")
    cells = torch.arange(width, device="cuda")[None, :] < hold[:, None]
    table[cells] = order[: sum(held)]
    st = {"case": case, "n_pages": n_pages, "table": table,
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "plan":
        rows = sum(max(d, 0) for d in delta) + case["pad"]
        free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        free[:spare] = order[sum(held):sum(held) + spare]
        st.update(delta=torch.tensor(delta, dtype=torch.int32, device="cuda"), free=free, rows=rows,
                  n_free=torch.tensor([spare], dtype=torch.int32, device="cuda"))
        return st

    dt, hq, hkv, d = DTYPES[case["dtype"]], case["q_heads"], case["kv_heads"], case["head_dim"]
    k = torch.empty((1, n_pages, hkv, page, d), dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty((1, n_pages, hkv, page, d), dtype=dt, device="cuda").normal_(generator=g)
    st.update(k=k, v=v, k_mean=None)
    if case["op"] == "write":
        # rows as a plan gives them: a request's new tokens follow what it holds
        cells = (torch.arange(width, device="cuda")[None, :] < torch.tensor(after, device="cuda")[:, None]) & ~cells
        table[cells] = order[sum(held): sum(held) + grow]
        rows = sum(delta) + case["pad"]
        new = torch.tensor(delta, device="cuda")
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), new)
        start = torch.cumsum(new, 0) - new
        pos = torch.arange(len(req), device="cuda") - start[req] + st["lens"].long()[req]
        slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        positions = torch.zeros(rows, dtype=torch.int32, device="cuda")
        slots[: len(req)] = (table.long()[req, pos // page] * page + pos % page).to(torch.int32)
        positions[: len(req)] = pos.to(torch.int32)
        st.update(slots=slots, positions=positions, qkv=normal(rows, (hq + 2 * hkv) * d).to(DTYPES[case["qkv"]]),
                  k_mean=k.float().mean(3).to(dt), q_out=torch.zeros((rows, hq * d), dtype=dt, device="cuda"))
    else:
        # queries from flat to peaked softmax (logits of spread 1 to 4)
        sharp = 1.0 + 3.0 * torch.rand((B, 1, 1), generator=g, device="cuda")
        st["q"] = (normal(B, hq, d) * sharp).to(dt)
        if case["op"] == "sparse":
            # pages of one scene share a direction, so that a page's mean says something of its keys
            k += (0.5 * normal(1, n_pages, hkv, 1, d)).to(dt)
            st["k_mean"] = k.float().mean(3).to(dt)
    return st


# ---------------------------------------------------------------------------------------
# one pass

def run(st):
    op = st["case"]["op"]
    return (_OWN if own else _PLAIN)[op](st, st["case"])


def _own_plan(st, case):
    h = st["pages"]
    h.R.rtvla_pages_plan(h.ctx, st["lens"], st["delta"], st["free"], st["n_free"], st["kv"], st["n_free_out"],
                         st["slots"], st["positions"], st["row_start"], st["rows"], torch.cuda.current_stream())
    return (st["lens_out"], st["table"], st["free"], st["n_free_out"], st["slots"], st["positions"],
            st["row_start"])


def _own_write(st, case):
    h = st["pages"]
    qkv_dtype = {"bf16": h.R.DTYPE_BF16, "f16": h.R.DTYPE_F16, "f32": h.R.DTYPE_F32}[case["qkv"]]
    h.R.rtvla_pages_write(h.ctx, 0, st["qkv"], qkv_dtype, st["slots"], st["positions"], len(st["slots"]), st["kv"],
                          st["q_out"], torch.cuda.current_stream())
    return st["q_out"], st["k"], st["v"], st["k_mean"]


def _own_attend(st, case):
    h = st["pages"]
    h.R.rtvla_pages_attend(h.ctx, 0, st["q"], st["kv"], None, 0, st["out"], torch.cuda.current_stream())
    return st["out"]


def _own_sparse(st, case):
    h, stream = st["pages"], torch.cuda.current_stream()
    h.R.rtvla_pages_select(h.ctx, 0, st["q"], st["kv"], case["budget"], case["keep_first"], case["keep_last"],
                           st["sel"], stream)
    h.R.rtvla_pages_attend(h.ctx, 0, st["q"], st["kv"], st["sel"], case["budget"], st["out"], stream)
    return st["sel"], st["out"]


def _plain_plan(st, case):
    page, rows = case["page"], st["rows"]
    lens, delta = st["lens"].long(), st["delta"].long()
    table, free = st["table"], st["free"]
    B, width = table.shape
    nf = st["n_free"].long()
    new = (lens + delta).clamp(min=0)
    held, after = (lens + page - 1) // page, (new + page - 1) // page
    grow, back = (after - held).clamp(min=0), (held - after).clamp(min=0)
    col = torch.arange(width, device="cuda")[None, :]
    # pages given back go on top of the free list, in request and page order
    gone = (col >= after[:, None]) & (col < held[:, None])
    cells = gone.nonzero()
    top = nf + torch.arange(len(cells), device="cuda")
    free[top] = table[cells[:, 0], cells[:, 1]]
    nf = nf + len(cells)
    # pages taken come from the top down
    want = (col >= held[:, None]) & (col < after[:, None])
    cells = want.nonzero()
    table[cells[:, 0], cells[:, 1]] = free[nf - 1 - torch.arange(len(cells), device="cuda")]
    nf = nf - len(cells)
    count = delta.clamp(min=0)
    row_start = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    row_start[1:] = torch.cumsum(count, 0)
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), count)
    pos = torch.arange(len(req), device="cuda") - row_start[req] + lens[req]
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    positions = torch.zeros(rows, dtype=torch.int32, device="cuda")
    slots[: len(req)] = (table[req, pos // page].long() * page + pos % page).to(torch.int32)
    positions[: len(req)] = pos.to(torch.int32)
    return (new.to(torch.int32), table, free, nf.to(torch.int32), slots, positions, row_start.to(torch.int32))


def _plain_write(st, case):
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    dt, half = DTYPES[case["dtype"]], case["head_dim"] // 2
    rows = len(st["slots"])
    freq = THETA ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / d)
    ang = st["positions"].double()[:, None] * freq
    c, s = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    x = st["qkv"].float().view(rows, hq + 2 * hkv, d)
    x1, x2 = x[:, : hq + hkv, :half], x[:, : hq + hkv, half:]
    y = torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1).to(dt)
    live = st["slots"] >= 0
    slot = st["slots"][live].long()
    pg, off = slot // page, slot % page
    st["k"][0, pg, :, off] = y[live, hq:]
    st["v"][0, pg, :, off] = x[live, hq + hkv:].to(dt)
    q_out = torch.where(live[:, None, None], y[:, :hq], st["q_out"].view(rows, hq, d))
    full = pg[off == page - 1]
    st["k_mean"][0, full] = st["k"][0, full].float().mean(2).to(dt)
    return q_out.reshape(rows, hq * d), st["k"], st["v"], st["k_mean"]


def _softmax_over(q, k, v, seen):
    """q [B][Hkv][G][d], k and v [B][Hkv][T][d], seen [B][1 or Hkv][T] -> [B][Hkv][G][d], fp32."""
    s = torch.matmul(q, k.transpose(-1, -2)) / q.shape[-1] ** 0.5
    s = s.masked_fill(~seen[:, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.masked_fill(~seen[..., None], 0.0))
    return torch.where(total > 0, o / total.clamp(min=1e-30), 0.0)


def _plain_attend(st, case):
    B, hkv, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    lens = st["lens"].long()
    idx = st["table"].clamp(min=0).long()
    T = idx.shape[1] * page
    k = st["k"][0][idx].transpose(1, 2).reshape(B, hkv, T, d).float()
    v = st["v"][0][idx].transpose(1, 2).reshape(B, hkv, T, d).float()
    seen = (torch.arange(T, device="cuda")[None, :] < lens[:, None])[:, None, :]
    q = st["q"].float().view(B, hkv, -1, d)
    return _softmax_over(q, k, v, seen).view(B, -1, d).to(st["q"].dtype)


def _plain_sparse(st, case):
    B, hkv, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    budget, first, last = case["budget"], case["keep_first"], case["keep_last"]
    lens = st["lens"].long()
    table = st["table"].clamp(min=0).long()
    W = table.shape[1]
    held = (lens + page - 1) // page
    # 64 bits: two pages' scores may lie next to each other
    qs = st["q"].double().view(B, hkv, -1, d).sum(2)
    score = torch.einsum("bhd,bwhd->bhw", qs, st["k_mean"][0][table].double())
    p = torch.arange(W, device="cuda")[None, :]
    kept = (p < first) | (p >= (held - last)[:, None]) | (held <= budget)[:, None]
    score = score.masked_fill(kept[:, None], float("inf")).masked_fill((p >= held[:, None])[:, None], float("-inf"))
    # a stable sort leaves ties in page order
    rank = torch.sort(score, dim=-1, descending=True, stable=True).indices
    n = held.clamp(max=budget)
    sel = torch.full((B, hkv, budget), W, dtype=torch.int64, device="cuda")
    m = min(budget, W)
    taken = torch.arange(m, device="cuda")[None, None, :] < n[:, None, None]
    sel[..., :m] = torch.where(taken, rank[..., :m], W)
    sel = torch.sort(sel, dim=-1).values
    live = sel < W
    sel = torch.where(live, sel, 0)
    phys = table[torch.arange(B, device="cuda")[:, None, None], sel]
    hh = torch.arange(hkv, device="cuda")[None, :, None]
    k = st["k"][0][phys, hh].reshape(B, hkv, budget * page, d).float()
    v = st["v"][0][phys, hh].reshape(B, hkv, budget * page, d).float()
    pos = sel[..., None] * page + torch.arange(page, device="cuda")
    seen = (live[..., None] & (pos < lens[:, None, None, None])).view(B, hkv, budget * page)
    out = _softmax_over(st["q"].float().view(B, hkv, -1, d), k, v, seen)
    return torch.where(live, sel, -1).to(torch.int32), out.view(B, -1, d).to(st["q"].dtype)


_OWN = {"plan": _own_plan, "write": _own_write, "attend": _own_attend, "sparse": _own_sparse}
_PLAIN = {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend, "sparse": _plain_sparse}


# ---------------------------------------------------------------------------------------
# the definition in 64 bits, request by request

def exact(case, seed):
    st = _inputs(case, seed)
    return {"plan": _exact_plan, "write": _exact_write, "attend": _exact_attend, "sparse": _exact_sparse}[case["op"]](
        st, case)


def _exact_plan(st, case):
    page, rows = case["page"], st["rows"]
    lens, delta = st["lens"].tolist(), st["delta"].tolist()
    table, free = st["table"].tolist(), st["free"].tolist()
    nf = int(st["n_free"])
    for b, (n, m) in enumerate(zip(lens, delta)):
        for i in range(_pages(max(n + m, 0), page), _pages(n, page)):
            free[nf] = table[b][i]
            nf += 1
    slots, positions, row_start = [], [], [0]
    for b, (n, m) in enumerate(zip(lens, delta)):
        for i in range(_pages(n, page), _pages(max(n + m, 0), page)):
            nf -= 1
            table[b][i] = free[nf]
        for t in range(n, n + m):
            slots.append(table[b][t // page] * page + t % page)
            positions.append(t)
        row_start.append(len(slots))
    pad = rows - len(slots)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    return (ints([max(n + m, 0) for n, m in zip(lens, delta)]), ints(table), ints(free), ints([nf]),
            ints(slots + [-1] * pad), ints(positions + [0] * pad), ints(row_start))


def _exact_write(st, case):
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    rows, half = len(st["slots"]), d // 2
    k, v, mean = st["k"].double(), st["v"].double(), st["k_mean"].double()
    z = st["qkv"].double().view(rows, hq + 2 * hkv, d)
    pair = torch.complex(z[:, : hq + hkv, :half], z[:, : hq + hkv, half:])
    freq = torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"),
                     -torch.arange(half, device="cuda", dtype=torch.float64) / half)
    turn = torch.polar(torch.ones((rows, half), dtype=torch.float64, device="cuda"),
                       torch.outer(st["positions"].double(), freq))
    pair = pair * turn[:, None, :]
    y = torch.cat((pair.real, pair.imag), -1)
    q_out = st["q_out"].double().view(rows, hq, d)
    slots = st["slots"].long()
    at = torch.nonzero(slots >= 0)[:, 0]
    q_out[at] = y[at, :hq]
    k = k.transpose(2, 3).reshape(-1, hkv, d)
    v = v.transpose(2, 3).reshape(-1, hkv, d)
    k[slots[at]] = y[at, hq:]
    v[slots[at]] = z[at, hq + hkv:]
    k = k.view(1, -1, page, hkv, d)
    for pg in (slots[at][slots[at] % page == page - 1] // page).tolist():
        mean[0, pg] = k[0, pg].sum(0) / page
    return (q_out.reshape(rows, hq * d), k.transpose(2, 3).contiguous(),
            v.view(1, -1, page, hkv, d).transpose(2, 3).contiguous(), mean)


def _one(q, k, v):
    """q [G][d], k and v [T][d] in 64 bits."""
    w = torch.softmax((q @ k.T) / q.shape[-1] ** 0.5, -1)
    return w @ v


def _exact_attend(st, case):
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    q = st["q"].double()
    out = torch.zeros_like(q).view(case["batch"], hkv, -1, d)
    for b, n in enumerate(st["lens"].tolist()):
        pg = st["table"][b, : _pages(n, page)].long()
        for h in range(hkv):
            if n:
                out[b, h] = _one(q[b].view(hkv, -1, d)[h], st["k"][0, pg, h].reshape(-1, d)[:n].double(),
                                 st["v"][0, pg, h].reshape(-1, d)[:n].double())
    return out.view_as(q)


def _exact_sparse(st, case):
    hkv, d, page, budget = case["kv_heads"], case["head_dim"], case["page"], case["budget"]
    q = st["q"].double()
    out = torch.zeros_like(q).view(case["batch"], hkv, -1, d)
    chosen = []
    for b, n in enumerate(st["lens"].tolist()):
        held = _pages(n, page)
        pg = st["table"][b, :held].long()
        for h in range(hkv):
            qh = q[b].view(hkv, -1, d)[h]
            sel = list(range(held))
            if held > budget:
                lo, hi = case["keep_first"], held - case["keep_last"]
                score = (st["k_mean"][0, pg, h].double() * qh.sum(0)).sum(-1).tolist()
                best = sorted(range(lo, hi), key=lambda i: (-score[i], i))[: budget - lo - (held - hi)]
                sel = sorted(list(range(lo)) + best + list(range(hi, held)))
            chosen.append(sel + [-1] * (budget - len(sel)))
            if n:
                at = torch.tensor(sel, device="cuda")
                pos = (at[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
                keys = st["k"][0, pg[at], h].reshape(-1, d)[pos < n].double()
                out[b, h] = _one(qh, keys, st["v"][0, pg[at], h].reshape(-1, d)[pos < n].double())
    sel = torch.tensor(chosen, dtype=torch.int32, device="cuda").view(case["batch"], hkv, budget)
    return sel, out.view_as(q)
