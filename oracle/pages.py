"""Plain fp64 numpy oracle of the paged KV cache (test infrastructure; shares no code with the
CUDA path).

Every function is a request-by-request loop over the definitions in include/rtvla.h: token t of a
request lives in slot table[b][t // page] * page + t % page; pages are popped from and pushed to a
stack in request and page order; attention is softmax(q K^T / sqrt(d)) V over the tokens held, in
logical order; a page's score is (sum of the group's query heads) . (mean key).
"""
from __future__ import annotations

import numpy as np

from . import model as _model


def pages_for(n: int, page: int) -> int:
    return -(-n // page)


def plan(lens, delta, table, free_pages, n_free, page, n_pages, n_rows):
    """One step's bookkeeping on copies.  Returns a dict of the results and the device errors."""
    lens, delta = [int(x) for x in lens], [int(x) for x in delta]
    table, free = np.array(table), np.array(free_pages)
    width, nf, err = table.shape[1], int(n_free), set()
    cap = width * page
    if not 0 <= nf <= n_pages:
        err.add("bounds")
        nf = min(max(nf, 0), n_pages)
    rows, start, alone = 0, [], []
    for n, d in zip(lens, delta):
        start.append(min(rows, n_rows))
        ok = 0 <= n <= cap
        if d > 0:
            rows += d
            ok = ok and min(max(n, 0), cap) + d <= cap and rows <= n_rows
        alone.append(not ok)
    start.append(min(rows, n_rows))
    if any(alone):
        err.add("bounds")
    lens = [min(max(n, 0), cap) for n in lens]
    after = [n if a else max(n + d, 0) for n, d, a in zip(lens, delta, alone)]
    for b, (n, m) in enumerate(zip(lens, after)):
        for i in range(pages_for(m, page), pages_for(n, page)):
            if not 0 <= table[b, i] < n_pages:  # pushed as it stands
                err.add("bounds")
            free[nf] = table[b, i]
            nf += 1
    slots, positions = np.full(n_rows, -1, np.int32), np.zeros(n_rows, np.int32)
    full = False
    for b, (n, m) in enumerate(zip(lens, after)):
        need = max(0, pages_for(m, page) - pages_for(n, page))
        if need and (full or need > nf):
            full = True
            after[b] = n
            err.add("no_pages")
            continue
        for i in range(need):
            nf -= 1
            table[b, pages_for(n, page) + i] = free[nf]
        for j, t in enumerate(range(n, m)):
            if not 0 <= table[b, t // page] < n_pages:  # a number that is no page: the row is skipped
                err.add("bounds")
                continue
            slots[start[b] + j] = table[b, t // page] * page + t % page
            positions[start[b] + j] = t
    return dict(lens=np.array(after, np.int32), table=table, free=free, n_free=nf, slots=slots,
                positions=positions, row_start=np.array(start, np.int32), err=err)


def rope(x, pos, theta):
    """x [..., d] rotated in pairs (i, i + d/2) by pos * theta^(-2i/d); theta 0: unchanged."""
    x = np.asarray(x, np.float64)
    if theta == 0:
        return x
    half = x.shape[-1] // 2
    z = x[..., :half] + 1j * x[..., half:]
    z = z * np.exp(1j * pos * theta ** (-np.arange(half) / half))
    return np.concatenate([z.real, z.imag], -1)


def write(qkv, slots, positions, n_q, n_kv, theta):
    """Rows [T][(Hq + 2 Hkv) d] -> (q [T][Hq][d], k [T][Hkv][d], v [T][Hkv][d]), fp64, unrounded."""
    T = len(slots)
    x = np.asarray(qkv, np.float64).reshape(T, n_q + 2 * n_kv, -1)
    y = np.stack([rope(x[t, : n_q + n_kv], int(positions[t]), theta) for t in range(T)]) if T else x[:, : n_q + n_kv]
    return y[:, :n_q], y[:, n_q:], x[:, n_q + n_kv:]


def keys_of(pool, table_row, n, h, page, picked=None):
    """The first n tokens' rows of KV head h in logical order (of the picked pages, in list order).

    pool [n_pages][Hkv][page][d]."""
    picked = range(pages_for(n, page)) if picked is None else picked
    rows = [pool[table_row[e], h, : min(page, n - e * page)] for e in picked]
    d = pool.shape[-1]
    return np.concatenate(rows).astype(np.float64) if rows else np.zeros((0, d))


def attend_one(q, k, v):
    """q [G][d], k, v [n][d] -> (out [G][d], sum_j p_j |v_j| [G][d], largest sum_i |q_i k_ji| / sqrt(d))."""
    q = np.asarray(q, np.float64)
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q), 0.0
    s = q @ k.T / np.sqrt(q.shape[-1])
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    size = float((np.abs(q) @ np.abs(k).T).max() / np.sqrt(q.shape[-1]))
    return p @ v, p @ np.abs(v), size


def scores(q, means):
    """q [G][d] (one KV head's query heads), means [pages][d] -> [pages]."""
    return np.asarray(means, np.float64) @ np.asarray(q, np.float64).sum(0)


def choose(score, held, budget, keep_first, keep_last):
    """Ascending list of the chosen pages of a request that holds `held` pages."""
    if held <= budget:
        return list(range(held))
    lo, hi = keep_first, held - keep_last
    best = sorted(range(lo, hi), key=lambda e: (-score[e], e))[: budget - keep_first - keep_last]
    return sorted(list(range(lo)) + best + list(range(hi, held)))


def prefix_step(weights, cfg, embed, K, V, pos):
    """One token through the prefix model: embed [Dp]; K, V: per layer the n keys and values held,
    [n][hd].  Returns (hidden [Dp] after the last layer, the token's keys [L][hd], values [L][hd]).

    The layer of oracle/model.py's prefix pass, for one query that sees every token held and itself.
    """
    x, ks, vs = np.asarray(embed, np.float64), [], []
    for l in range(cfg.n_layers):
        W = {n: np.asarray(weights[f"pf{l}.{n}"], np.float64)
             for n in ("ln1", "wq", "wk", "wv", "wo", "ln2", "wg", "wu", "wd")}
        n1 = _model.rms_normalize(x, cfg.rms_eps) * (1.0 + W["ln1"])
        q = rope((W["wq"] @ n1).reshape(cfg.n_q_heads, cfg.head_dim), pos, cfg.rope_theta)
        ks.append(rope(W["wk"] @ n1, pos, cfg.rope_theta))
        vs.append(W["wv"] @ n1)
        o = attend_one(q, np.vstack([K[l], ks[-1]]), np.vstack([V[l], vs[-1]]))[0]
        x = x + W["wo"] @ o.reshape(-1)
        n2 = _model.rms_normalize(x, cfg.rms_eps) * (1.0 + W["ln2"])
        x = x + W["wd"] @ (_model.gelu_tanh(W["wg"] @ n2) * (W["wu"] @ n2))
    return x, np.array(ks), np.array(vs)
