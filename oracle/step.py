"""Plain CPU oracle of a step with several new tokens per sequence.

TEST INFRASTRUCTURE ONLY.  Only the tests may import this module; the product
path never does.  It shares no code with the CUDA library.  Page by page, row
by row and token by token, in Python integers and numpy float64.

The sources ("DwarfStar 4 (DS4) - DeepSeek V4 Flash Inference Engine") define
no drafted tokens and no paging: the readings are the library's own and stated
in its header.  Segments are those of ``oracle.paged``.
"""

from __future__ import annotations

import numpy as np

from . import paged

D = 512
TREE_MOST = 128  # nodes of a tree that are seen


def page_tables(table, free, n_free, have, want, drop, page_rows, n_pages, n_slots):
    """Updates table (2-D array) and free (list of length n_pages) in place;
    returns (n_free, slots, first, n_short)."""
    B, width = table.shape
    n_free = min(max(n_free, 0), n_pages)
    plan = []
    for b in range(B):
        cap = width * page_rows
        h = min(max(int(have[b]), 0), cap)
        gone = 0 if drop is None else min(max(int(drop[b]), 0), h) // page_rows
        w = min(max(int(want[b]), 0), cap + gone * page_rows)
        held, need = -(-h // page_rows), max(-(-w // page_rows), gone)
        plan.append((h, w, gone, held, need))
        for i in list(range(gone)) + list(range(need, held)):
            if 0 <= table[b, i] < n_pages and n_free < n_pages:
                free[n_free] = int(table[b, i])
                n_free += 1
    slots, first, short = [], [0], 0
    for b, (h, w, gone, held, need) in enumerate(plan):
        row = [int(table[b, i]) for i in range(gone, min(held, need))]
        for _ in range(held, need):
            if n_free > 0:
                n_free -= 1
                row.append(free[n_free])
            else:
                short += 1
                row.append(-1)
        for i in range(max(held, need - gone)):
            table[b, i] = row[i] if i < len(row) else -1
        for r in range(h - gone * page_rows, w - gone * page_rows):
            page = row[r // page_rows]
            slots.append(page * page_rows + r % page_rows if 0 <= page < n_pages else -1)
        first.append(len(slots))
    slots = slots[:n_slots] + [-1] * (n_slots - len(slots))
    return n_free, np.array(slots, dtype=np.int32), np.minimum(first, n_slots).astype(np.int32), short


def spans(first, n_tok):
    """(start, tokens) of every sequence, clamped."""
    out = []
    for b in range(len(first) - 1):
        a = min(max(int(first[b]), 0), n_tok)
        out.append((a, min(max(int(first[b + 1]), a), n_tok) - a))
    return out


def parents_of(parent, start, n):
    """The parent of each of a sequence's nodes, -1 for a root."""
    if parent is None:
        return list(range(-1, n - 1))
    return [int(u) if 0 <= u < t else -1 for t, u in enumerate(parent[start:start + n])]


def accept(first, parent, token, target, prev, width):
    """(path lists, next) of every sequence."""
    paths, nxt = [], []
    for b, (start, n) in enumerate(spans(first, len(token))):
        up, at, path = parents_of(parent, start, n), -1, []
        want = None if prev is None else int(prev[b])
        while len(path) < width:
            fits = [t for t in range(n) if up[t] == at and (want is None or token[start + t] == want)]
            if not fits:
                break
            at = fits[0]
            path.append(at)
            want = int(target[start + at])
        paths.append(path)
        nxt.append(-1 if want is None else want)
    return paths, nxt


def commit(seg, geom, paths):
    """Moves the rows of the paths in place, one after the other."""
    n_pages, page_rows = seg["k"].shape[:2]
    cap = paged.capacity(seg)
    names = ["k"] if seg["v"] is seg["k"] else ["k", "v"]
    if seg.get("k_scale") is not None:
        names += ["k_scale"] if seg["v_scale"] is seg["k_scale"] else ["k_scale", "v_scale"]
    for b, path in enumerate(paths):
        base = max(int(geom[b][1]), 0)
        for i, u in enumerate(path):
            src, dst = base + int(u), base + i
            if u <= i or src >= cap:
                continue
            frm, to = int(seg["table"][b, src // page_rows]), int(seg["table"][b, dst // page_rows])
            if 0 <= frm < n_pages and 0 <= to < n_pages:
                for name in names:
                    seg[name][to, dst % page_rows] = seg[name][frm, src % page_rows]


def seen(shape, geom_b, parent, start, n, cap_raw, cap_comp):
    """Per token of a sequence: (raw rows, compressed rows) it sees, as lists of indices."""
    pos, n_raw, raw0, n_comp = (max(int(x), 0) for x in geom_b)
    n_raw, n_comp = min(n_raw, cap_raw), min(n_comp, cap_comp)
    up = parents_of(parent, start, n)
    ways, out = [], []
    for t in range(n):
        ways.append([t] + (ways[up[t]] if up[t] >= 0 else []))
        p = pos + len(ways[t]) - 1
        if parent is not None and t >= TREE_MOST:
            out.append(([], []))
            continue
        raw = [i for i in range(n_raw) if p - shape["window"] < raw0 + i <= p]
        raw += sorted(n_raw + u for u in ways[t][:shape["window"]] if n_raw + u < cap_raw)
        out.append((raw, list(range(min(n_comp, (p + 1) // shape["ratio"])))))
    return out


def attention(shape, geom, first, parent, q, raw, comp):
    """(o, lse, spread, reach, rows seen) per token, as ``oracle.paged.decode``;
    tokens of no sequence are NaN."""
    T = q.shape[0]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    spread, reach, count = np.zeros(q.shape), np.zeros(T), np.zeros(T, dtype=int)
    for b, (start, n) in enumerate(spans(first, T)):
        views = seen(shape, geom[b], parent, start, n, paged.capacity(raw), paged.capacity(comp))
        values = {}
        for seg, kind in ((raw, 0), (comp, 1)):
            most = max([max(v[kind], default=-1) + 1 for v in views], default=0)
            for which in "kv":
                values[kind, which] = paged.segment_rows(seg, b, most, which) if seg is not None and most else \
                    (np.zeros((most, D)), np.zeros(most, dtype=bool))
        for t, picks in enumerate(views):
            rows = {}
            for which in "kv":
                parts = []
                for kind in (0, 1):
                    x, have = values[kind, which]
                    i = np.array(picks[kind], dtype=int)
                    parts.append(x[i[have[i]]])
                rows[which] = np.concatenate(parts)
            k, v = rows["k"], rows["v"]
            at = start + t
            o[at], lse[at] = 0.0, -np.inf
            count[at] = len(k)
            if not len(k):
                continue
            qb = q[at].astype(np.float64)
            x = shape["scale"] * (qb @ k.T)
            m = x.max(1, keepdims=True)
            w = np.exp(x - m)
            l = w.sum(1, keepdims=True)
            o[at], spread[at] = (w @ v) / l, (w @ np.abs(v)) / l
            lse[at] = (m + np.log(l))[:, 0]
            reach[at] = abs(shape["scale"]) * (np.abs(qb) @ np.abs(k).T).max()
    return o, lse, spread, reach, count
