"""Rotary positions, attention weights of cached tokens and eviction plans in plain fp64 numpy: test infrastructure only.

It shares no code with the GPU path; rows and tokens are walked one at a time.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base, scaling="none", factor=1.0, context=1.0, low=0.0, high=1.0):
    """Radians per position of every pair."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        f = math.exp(-2.0 * i / rot * math.log(b))
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            wave = 2 * math.pi / f  # tokens of a turn
            turns = context / wave
            if turns <= low:
                f = f / factor
            elif turns < high:
                share = (turns - low) / (high - low)
                f = (1 - share) * f / factor + share * f
        out.append(f)
    return np.array(out)


def rotate(x, position, freq, layout, amplitude=1.0, inverse=False):
    """x [tokens][heads][D]: pairs of the first 2 len(freq) dimensions turned by position * freq."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    for t, p in enumerate(np.asarray(position).tolist()):
        for i, f in enumerate(freq):
            angle = p * f * (-1.0 if inverse else 1.0)
            a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = amplitude * math.cos(angle), amplitude * math.sin(angle)
            xa, xb = (np.asarray(x[t, :, d], dtype=np.float64) for d in (a, b))
            y[t, :, a] = xa * c - xb * s
            y[t, :, b] = xa * s + xb * c
    return y


def weights(q, keys, scale):
    """q [n][Hq][D], the queries of the last n of the cached keys [c][Hk][D]: what each key receives."""
    n, Hq, _ = q.shape
    c, Hk, _ = keys.shape
    out = np.zeros(c)
    for t in range(n):
        seen = c - n + t + 1
        for h in range(Hq):
            z = scale * (keys[:seen, h // (Hq // Hk)] @ q[t, h])
            e = np.exp(z - z.max())
            out[:seen] += e / e.sum()
    return out


def evict(page, n_pages, max_pages, kv_len, budget, score, token_pos, row_state, tables, free, n_free, sink, recent, max_moves):
    """The plan as lists per row; entries that it does not write are None.  A table's entries that are no pages of the cache:
    slot -1, the gap of such a pair keeps its token, and they do not get onto the stack."""
    B, width = score.shape
    rows, stack = [], [int(x) for x in free[:n_free]]
    most = min(width, max_pages * page)

    def status(i):
        c, b, (settled, gone) = int(kv_len[i]), int(budget[i]), (int(v) for v in row_state[i])
        if not (0 <= c <= most and 0 <= settled <= c and gone >= 0 and c + gone <= 2 ** 31 - 1):
            return "refused"
        if 0 <= b < c:
            return "kept, bad" if b < sink + recent or min(b, c - b) > max_moves else "cut"
        return "kept"

    states = [status(i) for i in range(B)]
    freed = sum(-(-int(kv_len[i]) // page) - -(-int(budget[i]) // page) for i in range(B) if states[i] == "cut")
    stack_ok = 0 <= n_free and n_free + freed <= n_pages
    for i in range(B):
        c, b = int(kv_len[i]), int(budget[i])
        settled, gone = (int(v) for v in row_state[i])
        if states[i] == "refused":
            rows.append(dict(kv_len=c, state=[settled, gone], score=[], pos=[], src=[], dst=[]))
            continue
        pos = [int(token_pos[i, j]) if j < settled else j + gone for j in range(c)]
        if states[i] != "cut" or not stack_ok:
            rows.append(dict(kv_len=c, state=[settled, gone], score=[float(s) for s in score[i, :c]], pos=pos, src=[], dst=[]))
            continue

        def rank(j):
            s = float(score[i, j])
            if pos[j] < sink or pos[j] >= c + gone - recent:
                return (0, 0.0, j)
            return (2, 0.0, j) if math.isnan(s) else (1, -s, j)

        kept = set(sorted(range(c), key=rank)[:b])
        movers, holes = [j for j in range(b, c) if j in kept], [j for j in range(b) if j not in kept]

        def slot(j):
            p = int(tables[i, j // page])
            return p * page + j % page if 0 <= p < n_pages else -1

        left = list(range(b))
        for j, h in zip(movers, holes):
            left[h] = j if slot(j) >= 0 and slot(h) >= 0 else h

        rows.append(dict(kv_len=b, state=[b, gone + c - b], score=[float(score[i, j]) for j in left], pos=[pos[j] for j in left],
                         src=[slot(j) for j in movers], dst=[slot(j) for j in holes]))
        stack += [int(p) for p in tables[i, -(-b // page):-(-c // page)] if 0 <= p < n_pages]
    return rows, stack if stack_ok else None, any(s in ("refused", "kept, bad") for s in states)
