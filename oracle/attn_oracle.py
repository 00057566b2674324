"""fp64 CPU oracle of the paged cache's bookkeeping, the attention over it and the verify over a tree of drafts -- TEST
INFRASTRUCTURE ONLY (the same rules as gdn_oracle: used by the tests alone, shares no code with the product path).

Attention of one query row over the keys it attends, straight from the definition:
    s_j = scale q.k_j,  o = sum_j e^(s_j) v_j / sum_j e^(s_j).
"""
from __future__ import annotations

import numpy as np

from . import gdn_oracle as orc

F64 = np.float64


def attend(q, k, v, seen, scale):
    """q (n,H_q,D), k and v (m,H_kv,D), seen (n,m) bool.  Returns (o, mag): the outputs (n,H_q,D) and the same
    averages of |v|, which bound how far roundings of the weights can move an output."""
    q, k, v = (np.asarray(t, F64) for t in (q, k, v))
    n, hq, D = q.shape
    g = hq // k.shape[1]
    o, mag = np.empty((n, hq, D)), np.empty((n, hq, D))
    for h in range(hq):
        s = np.where(seen, scale * (q[:, h] @ k[:, h // g].T), -np.inf)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        for i in range(n):  # keys that a row does not attend take no part, whatever they hold
            on = seen[i]
            o[i, h] = p[i, on] @ v[on, h // g]
            mag[i, h] = p[i, on] @ np.abs(v[on, h // g])
    return o, mag


def cached_rows(cache, table, count):
    """The first `count` tokens of one request: cache (n_pages,H_kv,P,D), table its page ids; (count,H_kv,D)."""
    P = cache.shape[2]
    return np.stack([cache[table[t // P], :, t % P] for t in range(count)]) if count else \
        np.zeros((0, cache.shape[1], cache.shape[3]), cache.dtype)


def prefill(q, k, v, cu, k_cache, v_cache, tables, ctx, scale):
    """Packed causal attention after cached prefixes; (o, mag) over all rows (NaN where no sequence has them)."""
    o, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for s in range(len(cu) - 1):
        a, b, c = int(cu[s]), int(cu[s + 1]), int(ctx[s])
        if a == b:
            continue
        kk, vv = (np.concatenate([cached_rows(pc, tables[s], c), t[a:b]]) for pc, t in ((k_cache, k), (v_cache, v)))
        seen = np.arange(c + b - a)[None, :] <= c + np.arange(b - a)[:, None]
        o[a:b], mag[a:b] = attend(q[a:b], kk, vv, seen, scale)
    return o, mag


def tree_paths(parent):
    """paths (n,n) bool: which nodes each node's path holds (its ancestors and itself)."""
    n = len(parent)
    on = np.zeros((n, n), bool)
    for j in range(n):
        at = j
        while at >= 0:
            on[j, at] = True
            at = int(parent[at])
    return on


def tree(q, k, v, parent, k_cache, v_cache, table, ctx, scale):
    """One row's tree: q (n,H_q,D), k and v (n,H_kv,D) of the drafts, parent (n,)."""
    kk, vv = (np.concatenate([cached_rows(pc, table, ctx), t]) for pc, t in ((k_cache, k), (v_cache, v)))
    seen = np.concatenate([np.ones((len(parent), ctx), bool), tree_paths(parent)], axis=1)
    return attend(q, kk, vv, seen, scale)


def verify_tree(geom, S0, hist0, x, a, b, conv_w, parent):
    """The gated delta rule over a tree of drafts of one slot: node j continues from node parent[j] (-1: from S0,
    hist0).  Returns (o (n,H,d_v), states (n,H,d_v,d_k), hists (n,W-1,C), depths (n,))."""
    out = []
    for j in range(x.shape[0]):
        p = int(parent[j])
        S, h, depth = (S0, hist0, 0) if p < 0 else out[p][1:]
        oj, S, h = orc.layer_sequence(geom, x[j:j + 1], a[j:j + 1], b[j:j + 1], conv_w, S, h)
        out.append((oj[0], S, h, depth + 1))
    return tuple(np.stack([e[i] for e in out]) for i in range(4))


def kv_plan(page, n_pages, max_pages, kv_len, new_len, free_pages, n_free, tables, max_tokens):
    """Block tables and slot maps by plain loops over requests and tokens (valid inputs, apart from a stack that runs
    out).  Returns a dict of the outputs; rows that cannot be served keep their length and get slots of -1."""
    tables, free = np.array(tables), np.array(free_pages)
    stack = [int(p) for p in free[:n_free]]
    ceil = lambda t: -(-int(t) // page)  # noqa: E731
    for c, n, row in zip(kv_len, new_len, tables):
        if n < 0:
            stack += [int(p) for p in row[:ceil(c)]]
    free[n_free:len(stack)] = stack[n_free:]
    slots, pos = np.full(max_tokens, -1, np.int32), np.zeros(max_tokens, np.int32)
    cu, out_len = [0], []
    demand = 0
    room = len(stack)
    for i, (c, n) in enumerate(zip(kv_len, new_len)):
        c, n = int(c), int(n)
        need = ceil(c + n) - ceil(c) if n > 0 else 0
        demand += need
        served = need == 0 or demand <= room
        if served:
            for e in range(need):
                tables[i, ceil(c) + e] = stack.pop()
        for t in range(max(n, 0)):
            at = cu[-1] + t
            if at < max_tokens:
                pos[at] = c + t
                if served:
                    slots[at] = tables[i, (c + t) // page] * page + (c + t) % page
        cu.append(cu[-1] + max(n, 0))
        out_len.append(c if not served else (0 if n < 0 else c + n))
    return dict(block_table=tables, free_pages=free, cu_new=np.minimum(cu, max_tokens).astype(np.int32), slot_map=slots,
                position=pos, kv_len_out=np.array(out_len, np.int32), n_free_out=len(stack))
