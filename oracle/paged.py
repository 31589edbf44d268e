"""Plain CPU oracle of the paged cache operators and of the norm.

TEST INFRASTRUCTURE ONLY.  Only the tests may import this module; the product
path never does.  It shares no code with the CUDA library.  All arithmetic is
float64 (numpy); whole numbers are exact.

A segment is a dict: ``k``, ``v`` [n_pages, page_rows, 512] (fp16 rows, or
uint8 E4M3 codes with ``k_scale`` / ``v_scale`` fp32 [n_pages, page_rows]) and
``table`` int [n_seq, max_pages].  Row i of sequence b is slot i % page_rows of
page table[b][i // page_rows]; an entry outside [0, n_pages) names no page and
its rows are invisible.  Visibility is that of ``oracle.mqa``: raw rows of the
sliding window, compressed rows whose span has ended.

Readings for the eviction and the norm ("DwarfStar 4 (DS4) - DeepSeek V4 Flash
Inference Engine" bounds neither the compressed rows nor defines the order of
the norm's roundings): they are the library's own and stated in its header.
"""

from __future__ import annotations

import numpy as np

from . import fp8

D = 512


def segment_rows(seg, b: int, n: int, which: str):
    """Rows 0 .. n-1 of sequence b: (float64 values [n, 512], present [n])."""
    pool, scale = seg[which], seg.get(which + "_scale")
    n_pages, page_rows = pool.shape[:2]
    out, present = np.zeros((n, D)), np.zeros(n, dtype=bool)
    for i in range(n):
        page, slot = int(seg["table"][b, i // page_rows]), i % page_rows
        if 0 <= page < n_pages:
            present[i] = True
            row = pool[page, slot]
            out[i] = row.astype(np.float64) if scale is None else \
                fp8.decode_table()[row] * np.float64(scale[page, slot])
    return out, present


def capacity(seg) -> int:
    return 0 if seg is None else seg["table"].shape[1] * seg["k"].shape[1]


def visible(shape, geom_b, cap_raw: int, cap_comp: int):
    """(first raw row, end of raw rows, compressed rows) the token sees."""
    pos, n_raw, raw0, n_comp = (max(int(x), 0) for x in geom_b)
    n_raw, n_comp = min(n_raw, cap_raw), min(n_comp, cap_comp)
    lo = min(max(pos - shape["window"] + 1 - raw0, 0), n_raw)
    hi = max(min(pos + 1 - raw0, n_raw), lo)
    return lo, hi, min(n_comp, (pos + 1) // shape["ratio"])


def seen_rows(shape, geom, b, raw, comp, which):
    lo, hi, nc = visible(shape, geom[b], capacity(raw), capacity(comp))
    parts, have = [np.zeros((0, D))], [np.zeros(0, dtype=bool)]
    if raw is not None and hi > lo:
        x, p = segment_rows(raw, b, hi, which)
        parts.append(x[lo:])
        have.append(p[lo:])
    if comp is not None and nc > 0:
        x, p = segment_rows(comp, b, nc, which)
        parts.append(x)
        have.append(p)
    have = np.concatenate(have)
    return np.concatenate(parts)[have]


def decode(shape, geom, q, raw, comp):
    """(o [B, 64, 512], lse [B, 64], spread): spread[b][h][d] = sum_j w_j |v_j|,
    the scale against which roundings of weights and values are measured, and
    the largest sum |q||k| of scale (for the rounding of the scores)."""
    B = q.shape[0]
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    spread, reach = np.zeros(q.shape), np.zeros(B)
    for b in range(B):
        k = seen_rows(shape, geom, b, raw, comp, "k")
        v = seen_rows(shape, geom, b, raw, comp, "v")
        if not len(k):
            continue
        qb = q[b].astype(np.float64)
        x = shape["scale"] * (qb @ k.T)
        m = x.max(1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(1, keepdims=True)
        o[b] = (p @ v) / l
        spread[b] = (p @ np.abs(v)) / l
        lse[b] = (m + np.log(l))[:, 0]
        reach[b] = abs(shape["scale"]) * (np.abs(qb) @ np.abs(k).T).max()
    return o, lse, spread, reach


def weights(shape, geom, q, comp, lse, before, decay):
    """Received weights [B, capacity]; NaN where the call writes nothing."""
    B, cap = q.shape[0], capacity(comp)
    out = np.full((B, cap), np.nan)
    for b in range(B):
        nc = visible(shape, geom[b], 0, cap)[2]
        k, have = segment_rows(comp, b, nc, "k")
        x = shape["scale"] * (q[b].astype(np.float64) @ k.T)
        ref = lse[b].astype(np.float64)[:, None]
        w = np.where(np.isneginf(ref), 0.0, np.exp(x - np.where(np.isneginf(ref), 0.0, ref))).sum(0)
        old = 0.0 if before is None else np.float64(np.float32(decay)) * before[b, :nc].astype(np.float64)
        out[b, :nc] = old + np.where(have, w, 0.0)
    return out


def evict(shape, geom, weights_, ids, n_keep: int, n_first: int, n_recent: int, cap: int):
    """Per sequence: (n', kept [n'] former slots)."""
    out = []
    for b in range(len(geom)):
        n = min(max(int(geom[b][3]), 0), cap)
        n_out = min(n, n_keep)
        ended = (max(int(geom[b][0]), 0) + 1) // shape["ratio"]

        def rank(j):
            i = j if ids is None else int(ids[b, j])
            w = float(weights_[b, j])
            if i < n_first or i >= ended - n_recent:
                return (0, 0.0, j)
            return (1, np.inf if np.isnan(w) else -w, j)
        keep = set(sorted(range(n), key=rank)[:n_out])
        kept = np.arange(n_out)
        gaps = [j for j in range(n_out) if j not in keep]
        movers = sorted(j for j in keep if j >= n_out)
        assert len(gaps) == len(movers)
        kept[gaps] = movers
        out.append((n_out, kept))
    return out


def move_rows(seg, b: int, kept) -> None:
    """Moves the kept rows of sequence b into their slots, in place."""
    n_pages, page_rows = seg["k"].shape[:2]
    names = ["k"] if seg["v"] is seg["k"] else ["k", "v"]
    if seg.get("k_scale") is not None:
        names += ["k_scale"] if seg["v_scale"] is seg["k_scale"] else ["k_scale", "v_scale"]
    for i, j in enumerate(kept):
        if i == j:
            continue
        to, frm = int(seg["table"][b, i // page_rows]), int(seg["table"][b, j // page_rows])
        if 0 <= to < n_pages and 0 <= frm < n_pages:
            for name in names:
                seg[name][to, i % page_rows] = seg[name][frm, j % page_rows]


def rmsnorm(x, weight, eps, residual=None):
    """(h, y) in float64."""
    h = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    ms = (h * h).sum(-1, keepdims=True) / h.shape[-1]
    return h, h / np.sqrt(ms + np.float64(np.float32(eps))) * weight.astype(np.float64)


def group_scales(y, group: int):
    """Largest magnitude / 448 per group of the last axis: [n, groups]."""
    width = y.shape[1]
    g = group or width
    return np.stack([np.abs(y[:, c:c + g]).max(1) for c in range(0, width, g)], 1) / 448.0


def e4m3_step(z):
    """Distance between neighbouring E4M3 numbers at z (2^-9 below 2^-6)."""
    a = np.abs(z)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    return np.exp2(np.minimum(e, 8.0) - 3)
