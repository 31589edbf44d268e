"""A step with several new tokens per sequence against the fp64 oracle (needs a GB300).

Page tables, accepted paths and moved rows are whole numbers and copies: bit for bit.
"""

import os
import re

import numpy as np
import pytest

from oracle import compressor, fp8, paged, step
from test_gpu_paged import (F16, check_decode, device_error_word_stays_clear, ds4a, host, poison, rows_on, shape_of,  # noqa: F401
                            torch, up)
from test_paged_oracle import make

pytestmark = pytest.mark.gpu

H, D = 64, 512


# ------------------------------------------------------------------ page tables

def page_case(rng, n_seq, page, rows, grow, dropped, spare, extra_width=2, absent=0.0):
    """Sequences with random lengths; a third grow, some shrink to nothing or a part, some stay."""
    have = rng.integers(0, rows + 1, n_seq)
    kind = rng.integers(0, 5, n_seq)
    want = np.where(kind < 3, have + rng.integers(0, grow + 1, n_seq), np.where(kind == 3, have, have // 3))
    want[kind == 4] = np.where(rng.random((kind == 4).sum()) < 0.5, 0, want[kind == 4])
    drop = rng.integers(0, np.maximum(have, 1) + page, n_seq) if dropped else None
    held = -(-have // page)
    width = int(max(1, -(-max(have.max(), want.max()) // page)) + extra_width)
    n_pages = max(1, int(held.sum()) + spare)
    order = rng.permutation(n_pages)
    table = rng.integers(-5, 0, (n_seq, width)).astype(np.int32)  # leftovers where no page is held
    at = 0
    for b in range(n_seq):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    table[:, :][(rng.random(table.shape) < absent)] = n_pages + 1
    free = np.full(n_pages, -7, dtype=np.int32)
    free[:n_pages - at] = order[at:]
    return have, want, drop, table, free, n_pages - at, n_pages


def run_pages(torch, ds4a, c, page, n_slots, stream=None):
    have, want, drop, table, free, n_free, n_pages = c
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    wide = torch.full((table.shape[0], table.shape[1] + 3), 99, dtype=torch.int32, device="cuda")
    t = wide[:, :table.shape[1]]
    t.copy_(i32(table))
    f, nf = i32(free), i32([n_free])
    slots, first, short = ds4a.page_tables(t, f, nf, i32(have), i32(want), page, drop=None if drop is None else i32(drop),
                                           n_slots=n_slots)
    assert (host(wide)[:, table.shape[1]:] == 99).all()
    return host(t), host(f), int(nf), host(slots), host(first), int(short)


@pytest.mark.parametrize("n_seq,page,rows,grow,spare", [
    (1, 64, 0, 1, 4), (1, 1, 5, 9, 20), (3, 64, 300, 40, 0), (64, 16, 200, 20, 90), (31, 7, 50, 60, 3),
    (1024, 16, 90, 40, 2000), (1025, 8, 30, 20, 100), (2500, 24, 60, 100, 20000), (2, 128, 5000, 9000, 200),
    (1100, 4, 500, 20, 100), (200, 4, 500, 20, 100)])
@pytest.mark.parametrize("dropped", [False, True])
def test_page_tables_match_the_oracle(torch, ds4a, n_seq, page, rows, grow, spare, dropped):
    rng = np.random.default_rng(n_seq * 1000 + page + dropped)
    c = page_case(rng, n_seq, page, rows, grow, dropped, spare, absent=0.02 if page == 7 else 0.0)
    new = int(np.maximum(c[1] - c[0], 0).sum())
    for n_slots in (new + 5, new // 2, 0):
        table, free = c[3].copy(), c[4].tolist()
        want = step.page_tables(table, free, c[5], c[0], c[1], c[2], page, c[6], n_slots)
        got = run_pages(torch, ds4a, c, page, n_slots)
        assert np.array_equal(got[0], table)
        assert np.array_equal(got[1], np.array(free, dtype=np.int32))
        assert got[2] == want[0] and got[5] == want[3]
        assert np.array_equal(got[3], want[1]) and np.array_equal(got[4], want[2])


def test_page_tables_of_any_numbers(torch, ds4a):
    """Negative, huge and contradicting numbers are clamped; a list that is full takes no more pages."""
    page, n_pages = 8, 12
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11], [0, 0, 0, 0]], dtype=np.int32)
    free = np.arange(n_pages, dtype=np.int32)
    for n_free in (-3, 0, 10, 12, 1 << 30):
        for have, want, drop in (([-5, 1 << 30, 32, 32], [7, -1, 1 << 30, 0], None),
                                 ([32, 32, 9, 32], [0, 0, 0, 0], [-1, 1 << 30, 8, 9]),
                                 ([32, 20, 9, 1], [1 << 30, 1 << 30, 100, 50], [32, 20, 9, 1])):
            c = (np.array(have), np.array(want), None if drop is None else np.array(drop), table, free, n_free, n_pages)
            t, f = table.copy(), free.tolist()
            want_ = step.page_tables(t, f, n_free, have, want, drop, page, n_pages, 40)
            got = run_pages(torch, ds4a, c, page, 40)
            assert np.array_equal(got[0], t) and np.array_equal(got[1], f) and got[2] == want_[0]
            assert np.array_equal(got[3], want_[1]) and np.array_equal(got[4], want_[2]) and got[5] == want_[3]


def test_page_tables_take_and_give_back(torch, ds4a):
    """Many calls in a row: no page is lost or held twice."""
    rng = np.random.default_rng(5)
    B, page, n_pages, width = 40, 16, 600, 40
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    table, free, n_free = i32(np.full((B, width), -1)), i32(rng.permutation(n_pages)), i32([n_pages])
    have = np.zeros(B, dtype=np.int64)
    for _ in range(12):
        want = rng.integers(0, 200, B)
        drop = rng.integers(0, np.maximum(have, 1))
        gone = drop // page
        want = np.maximum(want, gone * page)
        ds4a.page_tables(table, free, n_free, i32(have), i32(want), page, drop=i32(drop), n_slots=64)
        have = want - gone * page
        t, f = host(table), host(free)[:int(n_free)]
        held = np.concatenate([t[b, :-(-h // page)] for b, h in enumerate(have)])
        assert np.array_equal(np.sort(np.concatenate([held, f])), np.arange(n_pages))


def test_page_tables_of_the_most_slots(torch, ds4a):
    """As many slots as a 32-bit count names (8.6 GB of them): the blocks that fill them are counted in 64 bits."""
    c = (np.array([3, 0]), np.array([20, 5]), None, np.array([[0, -1, -1], [-1, -1, -1]], dtype=np.int32),
         np.array([1, 2, 3, 4, 0], dtype=np.int32), 4, 5)
    table, free = c[3].copy(), c[4].tolist()
    want = step.page_tables(table, free, c[5], c[0], c[1], None, 8, c[6], 30)
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    slots = torch.empty(2 ** 31 - 1, dtype=torch.int32, device="cuda")
    slots[-2000:] = 7
    t, f, nf = i32(c[3]), i32(c[4]), i32([c[5]])
    _, first, short = ds4a.page_tables(t, f, nf, i32(c[0]), i32(c[1]), 8, slots=slots)
    assert np.array_equal(host(t), table) and np.array_equal(host(f), free) and int(nf) == want[0]
    assert np.array_equal(host(slots[:30]), want[1]) and host(first).tolist() == want[2].tolist() and int(short) == want[3]
    assert all(bool((part == -1).all()) for part in slots[22:].split(1 << 28))


# ------------------------------------------------------------------ acceptance

def tree_of(rng, n, chain, wide=8):
    if chain:
        return np.arange(-1, n - 1)
    t = np.arange(n)
    p = t - 1 - (rng.random(n) * np.minimum(t, wide)).astype(int)
    p[rng.random(n) < 0.1] = -1
    return np.maximum(p, -1)


def accept_case(rng, counts, chain, tokens=3):
    """Few different tokens: paths of every length, and siblings that hold the same one."""
    first = np.concatenate([[0], np.cumsum(counts)])
    parent = None if chain else np.concatenate([tree_of(rng, n, False) for n in counts] + [np.zeros(0, int)])
    n = first[-1]
    return first, parent, rng.integers(0, tokens, n), rng.integers(0, tokens, n), rng.integers(0, tokens, len(counts))


def check_accept(torch, ds4a, first, parent, token, target, prev, width):
    i32 = lambda a: None if a is None else up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    B = len(first) - 1
    wide = torch.full((B, width + 2), 77, dtype=torch.int32, device="cuda")
    path, count, nxt = ds4a.tree_accept(i32(first), i32(token), i32(target), parent=i32(parent), prev=i32(prev),
                                        path=wide[:, :width])
    paths, want = step.accept(first, parent, token, target, prev, width)
    assert host(nxt).tolist() == want and host(count).tolist() == [len(p) for p in paths]
    assert host(path).tolist() == [p + [-1] * (width - len(p)) for p in paths]
    assert (host(wide)[:, width:] == 77).all()


@pytest.mark.parametrize("counts", [[1], [8], [0], [5, 0, 33, 128, 1], [129, 200, 64], [700, 3], [2] * 300])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("tokens", [1, 2, 50])
def test_accept_matches_the_oracle(torch, ds4a, counts, chain, tokens):
    rng = np.random.default_rng(sum(counts) + tokens)
    first, parent, token, target, prev = accept_case(rng, counts, chain, tokens)
    for p in (prev, None):
        for width in (max(counts) + 1, 3):
            check_accept(torch, ds4a, first, parent, token, target, p, width)


def test_accept_of_any_parents_and_ranges(torch, ds4a):
    """Entries that are no earlier node are roots; ranges are clamped to the tokens."""
    rng = np.random.default_rng(8)
    n = 60
    parent = rng.integers(-3, 70, n)
    parent[3], parent[4] = 3, 1 << 30
    token, target = rng.integers(0, 2, n), rng.integers(0, 2, n)
    for first in ([0, 30, 60], [-5, 40, 1 << 30], [20, 10, 60], [60, 60, 60]):
        check_accept(torch, ds4a, first, parent, token, target, np.array([1, 0]), 20)


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("f8,shared,page,counts,pad", [
    (False, True, 16, [8], 0), (False, False, 64, [16, 1, 0, 30], 0), (True, False, 7, [64, 20, 3], 16),
    (True, True, 32, [128, 65], 0), (False, False, 1, [70, 200], 8)])
def test_commit_matches_the_oracle(torch, ds4a, f8, shared, page, counts, pad):
    rng = np.random.default_rng(page + len(counts))
    n = len(counts)
    n_raw = rng.integers(0, 140, n)
    seg = make(rng, n, (n_raw + counts).tolist(), page, f8, shared, absent=((n - 1, 0),) if page == 7 else ())
    paths = [np.flatnonzero(rng.random(c) < 0.4).tolist() for c in counts]
    paths[0] = list(range(0, counts[0], 2))
    geom = [(5, int(r), 0, 0) for r in n_raw]
    width = max(counts) + 1
    table = np.full((n, width + 3), -1, dtype=np.int32)
    for b, p in enumerate(paths):
        table[b, :len(p)] = p
    rows = rows_on(torch, ds4a, seg, pad_row=pad)
    before = {k: (v.copy() if v is not None else None) for k, v in seg.items()}
    if shared:
        before["v"], before["v_scale"] = before["k"], before.get("k_scale")
    step.commit(before, geom, paths)
    ds4a.commit_paged(rows, up(torch, np.array(geom, dtype=np.int32)), up(torch, table)[:, :width],
                      up(torch, np.array([len(p) for p in paths], dtype=np.int32)))
    for name in ("k", "v"):
        got = host(getattr(rows, name)).view(np.uint8)
        assert np.array_equal(got, np.ascontiguousarray(before[name]).view(np.uint8)), name
        if f8:
            assert np.array_equal(host(getattr(rows, name + "_scale")), before[name + "_scale"])


def test_commit_of_any_numbers(torch, ds4a):
    """Rows behind the table, negative and repeated nodes: nothing outside the sequence's rows is touched."""
    rng = np.random.default_rng(3)
    seg = make(rng, 3, [40, 40, 40], 8, False, False)
    rows = rows_on(torch, ds4a, seg)
    geom = np.array([(0, 30, 0, 0), (0, -9, 0, 0), (0, 1 << 30, 0, 0)], dtype=np.int32)
    path = np.array([[2, 5, 9, 100, 1 << 30], [-4, -1, 2, 3, 4], [1, 2, 3, 4, 5]], dtype=np.int32)
    ds4a.commit_paged(rows, up(torch, geom), up(torch, path), up(torch, np.array([99, 5, 5], dtype=np.int32)))
    step.commit(seg, geom, [[2, 5, 9, 100, 1 << 30], [-4, -1, 2, 3, 4], [1, 2, 3, 4, 5]])
    for name in ("k", "v"):
        assert np.array_equal(host(getattr(rows, name)), seg[name])


# ------------------------------------------------------------------ attention of several new tokens
# Tolerances: as for one token (test_gpu_paged.py): a rounding of the weights and one of the output to fp16, the
# scores' fp32 sums, and fp32 sums of the weights.

def tree_case(rng, counts, comp_rows, ratio, page, f8=False, shared=True, window=128, absent=(), chain=False,
              extra=1, wide=8):
    """Sequences whose new tokens come right after the cached rows; NaN wherever no row is in use."""
    geom, raw_rows = [], []
    for c, n in zip(comp_rows, counts):
        pos = c * ratio + min(extra, ratio - 1)
        first = max(0, pos + 1 - window) // page * page
        geom.append((pos, pos - first, first, (pos + n) // ratio if chain else c))
        raw_rows.append(pos - first + n)
    have_comp = [g[3] for g in geom]
    comp = make(rng, len(counts), have_comp, page, f8, shared, absent)
    raw = make(rng, len(counts), raw_rows, page, f8, shared)
    poison(comp, have_comp)
    poison(raw, raw_rows)
    first = np.concatenate([[0], np.cumsum(counts)])
    parent = None if chain else np.concatenate([tree_of(rng, n, False, wide) for n in counts] + [np.zeros(0, int)])
    q = rng.standard_normal((first[-1], H, D)).astype(np.float16)
    return geom, first, parent, q, raw, comp


def check_tree(got_o, got_lse, want):
    o, lse, spread, reach, count = want
    check_decode(got_o, got_lse, (o, lse, spread, reach), count)


def run_tree(torch, ds4a, shape, geom, first, parent, q, raw, comp, **kw):
    i32 = lambda a: None if a is None else up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    o, lse = ds4a.attn_tree_paged(shape, i32(geom), i32(first), up(torch, q), raw, comp, parent=i32(parent),
                                  want_lse=True, **kw)
    return host(o), host(lse)


TREES = [
    # counts, compressed rows, ratio, page, f8, shared, chain, window
    ([1], [0], 4, 16, False, True, False, 128),
    ([2], [3], 4, 16, False, False, True, 128),
    ([8], [256], 128, 64, False, True, False, 128),
    ([8], [256], 128, 64, True, True, False, 128),
    ([3, 1, 7, 0, 16], [40, 500, 0, 9, 1100], 4, 16, False, False, False, 128),
    ([3, 1, 7, 0, 16], [40, 500, 0, 9, 1100], 4, 16, True, False, False, 128),
    ([64, 13, 128], [700, 64, 300], 4, 32, False, True, False, 128),
    ([64, 13, 128], [700, 64, 300], 4, 32, True, True, False, 128),
    ([33, 20], [200, 90], 1, 24, False, True, False, 7),
    ([40, 21], [517, 255], 1, 8, False, False, True, 128),
    ([150, 299], [10, 40], 4, 100, False, True, True, 128),
    ([61, 200, 5], [300, 20, 2], 4, 64, True, False, True, 33),
    ([5, 4], [1024, 2000], 4, 128, False, False, False, 1),
    ([17] * 20, list(range(0, 400, 20)), 4, 16, False, True, False, 128),
    ([2] * 90, [30] * 90, 128, 7, True, True, True, 128),
    ([30, 9], [530, 300], 4, 12, False, False, False, 128),
    ([64, 100], [900, 511], 4, 20, True, False, False, 50),
    ([64, 100], [900, 511], 4, 40, True, False, True, 50),
    ([31, 128], [1500, 256], 2, 56, False, True, False, 128),
]


@pytest.mark.parametrize("k", range(len(TREES)))
def test_tree_matches_the_oracle(torch, ds4a, k):
    counts, rows, ratio, page, f8, shared, chain, window = TREES[k]
    rng = np.random.default_rng(100 + k)
    geom, first, parent, q, raw, comp = tree_case(rng, counts, rows, ratio, page, f8, shared, window, chain=chain)
    shape = shape_of(ratio, window)
    want = step.attention(shape, geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape, geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("chain", [False, True])
def test_tree_long_ragged_batches(torch, ds4a, f8, chain):
    """Many tiles in a row, of every kind, and sequences cut over several groups of SMs."""
    rng = np.random.default_rng(7 + f8)
    counts, rows = [9, 2, 30, 1, 5, 12], [9000, 40, 2500, 6000, 1, 700]
    geom, first, parent, q, raw, comp = tree_case(rng, counts, rows, 4, 64, f8, not chain, chain=chain)
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, r, c)
    check_tree(*got, want)
    for _ in range(3):
        again = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, r, c)
        assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


@pytest.mark.parametrize("f8", [False, True])
def test_tree_absent_pages(torch, ds4a, f8):
    rng = np.random.default_rng(21)
    geom, first, parent, q, raw, comp = tree_case(rng, [6, 9], [600, 90], 4, 32, f8, False,
                                                  absent=((0, 0), (0, 7), (0, 8), (1, 2)))
    raw["table"][0, 1] = -1
    raw["table"][1, raw["table"].shape[1] - 1] = 1 << 30  # the new rows of a sequence, perhaps
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("f8", [False, True])
def test_tree_strides_and_untouched_tokens(torch, ds4a, f8):
    """Padded pools, tokens and outputs; tokens behind the last sequence keep what they held."""
    rng = np.random.default_rng(22)
    geom, first, parent, q, raw, comp = tree_case(rng, [3, 10], [300, 31], 4, 16, f8, False)
    n, T = int(first[-1]), int(first[-1]) + 5
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    big_q = torch.full((T, H * D + 24), float("nan"), dtype=torch.float16, device="cuda")
    big_o = torch.full((T, H * D + 8), 7.0, dtype=torch.float16, device="cuda")
    qv = big_q.as_strided((T, H, D), (H * D + 24, D, 1))
    ov = big_o.as_strided((T, H, D), (H * D + 8, D, 1))
    qv[:n] = up(torch, q)
    lse = torch.full((T, H), 5.0, device="cuda")
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    ds4a.attn_tree_paged(shape_of(4), i32(geom), i32(first), qv, rows_on(torch, ds4a, raw, 16, 64),
                         rows_on(torch, ds4a, comp, 32, 128), parent=i32(np.concatenate([parent, np.zeros(5)])), out=ov,
                         lse=lse)
    check_tree(host(ov)[:n], host(lse)[:n], want)
    assert (host(big_o)[n:] == 7).all() and (host(big_o)[:, H * D:] == 7).all() and (host(lse)[n:] == 5).all()


@pytest.mark.parametrize("raw_page,comp_page", [(8, 64), (64, 8), (16, 24), (256, 16), (7, 64), (64, 7), (40, 128), (1, 1)])
@pytest.mark.parametrize("f8", [False, True])
def test_tree_pages_of_two_sizes(torch, ds4a, raw_page, comp_page, f8):
    """Raw and compressed rows in pages of sizes of their own; K and V one pool in one segment and two in the other."""
    rng = np.random.default_rng(raw_page + comp_page)
    geom, first, parent, q, raw, _ = tree_case(rng, [5, 40, 1], [530, 70, 0], 4, raw_page, f8, True)
    counts = [g[3] for g in geom]
    comp = make(rng, 3, counts, comp_page, f8, False)
    poison(comp, counts)
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


def test_tree_of_more_nodes_than_are_seen(torch, ds4a):
    """Nodes behind the 128th see no row; a chain of as many does."""
    rng = np.random.default_rng(23)
    geom, first, parent, q, raw, comp = tree_case(rng, [131, 4], [50, 6], 4, 16)
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    assert (want[0][128:131] == 0).all() and np.isneginf(want[1][128:131]).all()
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("chain", [False, True])
def test_tree_of_any_numbers(torch, ds4a, chain):
    """Parents that are no earlier node, new rows behind the table, ranges and geometry out of bounds, segments
    without rows: what the oracle, which goes by the definition, says."""
    rng = np.random.default_rng(24)
    geom, first, parent, q, raw, comp = tree_case(rng, [12, 20, 3], [40, 90, 2], 4, 16, chain=chain)
    if not chain:
        parent = rng.integers(-4, 25, 35)
        parent[5] = 1 << 30
    geom[0] = (geom[0][0], raw["table"].shape[1] * 16 - 4, 0, 1 << 30)  # most new rows behind the table
    geom[1] = (-5, -7, -3, -1)
    for seg in (raw, comp):  # every row may be read now
        seg["k"][np.isnan(seg["k"])] = 1.0
        seg["table"][seg["table"] < 0] = 0
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    for f in (first, [-9, 12, 32, 1 << 30], [0, 0, 35, 35], [12, 12, 12, 12]):
        for rr, cc, ro, co in ((r, c, raw, comp), (r, None, raw, None), (None, c, None, comp), (None, None, None, None)):
            want = step.attention(shape_of(4), geom, f, parent, q, ro, co)
            mine = ~np.isnan(want[0][:, 0, 0])
            o, lse = run_tree(torch, ds4a, shape_of(4), geom, f, parent, q, rr, cc)
            check_tree(o[mine], lse[mine], tuple(x[mine] for x in want))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("chain", [False, True])
def test_tree_bad_rows_spoil_their_tokens_only(torch, ds4a, f8, chain):
    """A row that holds NaN or infinities (as K, as V, or both) reaches the tokens that see it, and no others."""
    rng = np.random.default_rng(25)
    counts = [12, 40]
    geom, first, parent, q, raw, comp = tree_case(rng, counts, [150, 300], 4 if chain else 128, 16, f8, False, chain=chain)
    want = step.attention(shape_of(4 if chain else 128), geom, first, parent, q, raw, comp)
    for node, which, value in ((3, "k", np.nan), (7, "v", np.nan), (11, "v", np.inf), (0, "v", -np.inf)):
        for b, cached in ((0, False), (1, False), (1, True)):
            seg = {k: (None if x is None else x.copy()) for k, x in raw.items()}
            row = geom[b][1] - 100 + node if cached else geom[b][1] + node  # (a cached row leaves a run's window)
            page, slot = seg["table"][b, row // 16], row % 16
            bad = 0x7F if f8 else value
            seg[which][page, slot, 5] = bad
            seg[which][page, slot, 300] = bad
            o, lse = run_tree(torch, ds4a, shape_of(4 if chain else 128), geom, first, parent, q,
                              rows_on(torch, ds4a, seg), rows_on(torch, ds4a, comp))
            views = step.seen(shape_of(4 if chain else 128), geom[b], parent, int(first[b]), counts[b], 1 << 20, 1 << 20)
            hit = np.zeros(len(q), dtype=bool)
            hit[first[b]:first[b + 1]] = [row in v[0] for v in views]
            assert hit.any() and not hit.all()
            check_tree(o[~hit], lse[~hit], tuple(x[~hit] for x in want))
            assert not np.isfinite(o[hit][:, :, 5]).any() and not np.isfinite(o[hit][:, :, 300]).any()
            if which == "k":
                assert np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
            else:
                assert np.isfinite(lse[hit]).all()


@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_tree_bad_scales_spoil_their_tokens_only(torch, ds4a, page, value):
    """A scale that is not finite: of K, of V, of a new row that some see, of a compressed row that all see."""
    rng = np.random.default_rng(33)
    counts, ratio = [12, 40], 128
    geom, first, parent, q, raw, comp = tree_case(rng, counts, [150, 300], ratio, page, True, False)
    shape = shape_of(ratio)
    want = step.attention(shape, geom, first, parent, q, raw, comp)
    for which, b, node in (("v", 0, 4), ("v", 1, 9), ("v", 1, None), ("k", 0, 5)):
        mine = {n: {k: (None if x is None else x.copy()) for k, x in s.items()} for n, s in (("raw", raw), ("comp", comp))}
        row = 30 if node is None else geom[b][1] + node
        seg = mine["comp" if node is None else "raw"]
        seg[which + "_scale"][seg["table"][b, row // page], row % page] = value
        o, lse = run_tree(torch, ds4a, shape, geom, first, parent, q, rows_on(torch, ds4a, mine["raw"]),
                          rows_on(torch, ds4a, mine["comp"]))
        views = step.seen(shape, geom[b], parent, int(first[b]), counts[b], 1 << 20, 1 << 20)
        hit = np.zeros(len(q), dtype=bool)
        hit[first[b]:first[b + 1]] = [row in v[1 if node is None else 0] for v in views]
        assert hit.any() and not hit.all()
        check_tree(o[~hit], lse[~hit], tuple(x[~hit] for x in want))
        if which == "k" and value == np.inf:  # a score of -inf is a weight of 0
            dots = q[hit].astype(np.float64) @ fp8.decode_table()[seg["k"][seg["table"][b, row // page], row % page]]
            assert (np.isnan(o[hit]).all(2) == (dots > 0)).all() and (dots > 0).any()
            continue
        assert np.isnan(o[hit]).all()
        if which == "v":  # the weights are what they were
            lse_ = lse.copy()
            o[hit] = want[0][hit]
            check_tree(o, lse_, want)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [16, 7])
def test_tree_first_tile_without_rows(torch, ds4a, f8, page):
    """The pages of a sequence's first compressed rows are absent, so that nothing is seen there; then of all."""
    rng = np.random.default_rng(31)
    geom, first, parent, q, raw, comp = tree_case(rng, [5, 4, 2], [700, 600, 40], 4, page, f8, False)
    for b, gone in ((0, 560 // page), (1, 100000), (2, 100000)):
        comp["table"][b, :gone] = -1
    raw["table"][2] = 1 << 20
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    assert (want[4][9:] == 0).all() and (want[4][:9] > 100).all()
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


def test_tree_pages_past_32_bit_offsets(torch, ds4a):
    """A pool of over 4 GB: rows at its far end."""
    rng = np.random.default_rng(26)
    page, n_pages = 64, 70000
    pool = torch.zeros((n_pages, page, D), dtype=torch.float16, device="cuda")
    counts, rows = [5, 8], [400, 130]
    geom, first, parent, q, raw, comp = tree_case(rng, counts, rows, 4, page)
    far = {}
    for name, seg, base in (("raw", raw, n_pages - 40), ("comp", comp, n_pages - 80)):
        pool[base:base + len(seg["k"])] = up(torch, seg["k"])
        far[name] = ds4a.PagedRows(pool, None, up(torch, np.where(seg["table"] >= 0, seg["table"] + base, -1).astype(np.int32)))
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, far["raw"], far["comp"])
    check_tree(*got, want)


@pytest.mark.parametrize("exponent", [-60, -12, 0, 12])
def test_tree_e4m3_scales_of_any_size(torch, ds4a, exponent):
    """V scales far from 1: the output scales with them."""
    rng = np.random.default_rng(27)
    geom, first, parent, q, raw, comp = tree_case(rng, [7, 4], [300, 77], 4, 16, True, False)
    for seg in (raw, comp):
        live = np.isfinite(seg["v_scale"])
        seg["v_scale"][live] *= np.float32(2.0) ** exponent
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("page", [64, 8, 12])
def test_tree_e4m3_value_scales_of_zero(torch, ds4a, page):
    """Rows with weight and no value, whatever their codes, in tiles that are seen in full and at their edges."""
    rng = np.random.default_rng(34)
    geom, first, parent, q, raw, comp = tree_case(rng, [7, 12], [1100, 300], 4, page, True, False)
    for seg, rows in ((raw, [g[1] + n for g, n in zip(geom, (7, 12))]), (comp, [1100, 300])):
        for b, n in enumerate(rows):
            gone = rng.random(n) < 0.1
            gone[n // 2:n // 2 + 70] = True
            for i in np.flatnonzero(gone):
                seg["v_scale"][seg["table"][b, i // page], i % page] = rng.choice([0.0, 2.0 ** -60])
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("f8", [False, True])
def test_tree_large_scores_move_the_reference(torch, ds4a, f8):
    """Scores that grow along the rows, by far more than an exponent holds."""
    rng = np.random.default_rng(28)
    geom, first, parent, q, raw, comp = tree_case(rng, [6], [3000], 4, 64, f8, False)
    q = (q.astype(np.float32) * 2).astype(np.float16)
    if not f8:
        grow = np.linspace(0.1, 12, 3000)
        for i in range(3000):
            comp["k"][comp["table"][0, i // 64], i % 64] *= np.float16(grow[i])
    else:
        for i in range(3000):
            comp["k_scale"][comp["table"][0, i // 64], i % 64] *= np.float32(0.1 + i / 250)
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("below", [6, 12, 18, 24])
def test_tree_of_a_long_tail_under_one_row(torch, ds4a, below):
    """65,000 rows 2^-below under a single one: each rounds to little, together they count."""
    rng = np.random.default_rng(29)
    n, page = 65000, 64
    geom, first, parent, q, raw, comp = tree_case(rng, [2], [n], 1, page, False, False)
    axis = np.zeros(D, dtype=np.float16)
    axis[0] = 16.0
    q[:] = axis
    raw["k"][np.isfinite(raw["k"])] = 0
    raw["k"][:, :, 0] = np.where(np.isfinite(raw["k"][:, :, 0]), -64.0, np.nan)  # far below all others
    scale = 1.0 / np.sqrt(512.0)
    low = -below * np.log(2.0) / (16.0 * scale)
    comp["k"][np.isfinite(comp["k"])] = 0
    comp["k"][:, :, 0] = np.where(np.isfinite(comp["k"][:, :, 0]), low, np.nan)
    comp["k"][comp["table"][0, 300], 5, 0] = 0.0
    comp["v"][np.isfinite(comp["v"])] = 1.0
    comp["v"][comp["table"][0, 300], 5] = -1.0
    want = step.attention(shape_of(1), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(1), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("f8", [False, True])
def test_tree_units_of_a_single_tile(torch, ds4a, f8):
    """Items that are one tile each, many to a pair of SMs: a head's maximum and its sum, of sizes far apart between
    heads, pass between the same four warps with nothing else in between.  Every call gives the oracle's values."""
    rng = np.random.default_rng(34)
    counts = [int(x) for x in rng.integers(1, 5, 260)]
    rows = [int(x) for x in rng.integers(0, 100, 260)]
    geom, first, parent, q, raw, comp = tree_case(rng, counts, rows, 128, 16, f8, True, window=64)
    q = (q.astype(np.float32) * np.geomspace(0.1, 10, H)[rng.permutation(H)][None, :, None]).astype(np.float16)
    shape = shape_of(128, 64)
    want = step.attention(shape, geom, first, parent, q, raw, comp)
    assert (want[4] + 64 <= 256).all()  # one tile to a unit
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    args = (shape, i32(geom), i32(first), up(torch, q), rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    o, lse = ds4a.attn_tree_paged(*args, parent=i32(parent), want_lse=True)
    check_tree(host(o), host(lse), want)
    for _ in range(200):
        again = ds4a.attn_tree_paged(*args, parent=i32(parent), want_lse=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_tree_of_more_sequences_than_a_plan_holds(torch, ds4a):
    """1,300 trees: where units begin is kept in the workspace, and units are counted in several rounds."""
    rng = np.random.default_rng(35)
    counts = [int(x) for x in rng.integers(0, 5, 1300)]
    rows = [int(x) for x in rng.integers(0, 9, 1300)]
    geom, first, parent, q, raw, comp = tree_case(rng, counts, rows, 4, 8, window=6)
    assert sum((n + 1) // 2 for n in counts) > 1024
    want = step.attention(shape_of(4, 6), geom, first, parent, q, raw, comp)
    got = run_tree(torch, ds4a, shape_of(4, 6), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    check_tree(*got, want)


@pytest.mark.parametrize("chain", [False, True])
def test_tree_of_more_units_than_blocks_have_threads(torch, ds4a, chain):
    """66,000 tokens in 33,000 pairs, over 1,024 to a block of the plan: 600 sequences alike, whose results have the same
    bits, since a pair's rows are one tile that no border cuts."""
    rng = np.random.default_rng(36)
    n_seq, n = 600, 110
    geom, _, parent, q, raw, comp = tree_case(rng, [n], [9], 4, 16, window=24, chain=chain)
    want = step.attention(shape_of(4, 24), geom, [0, n], parent, q, raw, comp)
    assert n_seq * (n // 2) > 32 * 1024 and want[4].max() + n < 256
    for seg in (raw, comp):
        seg["table"] = np.repeat(seg["table"], n_seq, axis=0)
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    o, lse = ds4a.attn_tree_paged(shape_of(4, 24), i32(geom * n_seq), i32(np.arange(n_seq + 1) * n),
                                  up(torch, q).repeat(n_seq, 1, 1), rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp),
                                  parent=None if chain else i32(np.tile(parent, n_seq)), want_lse=True)
    check_tree(host(o[:n]), host(lse[:n]), want)
    assert all(torch.equal(o[i:i + n], o[:n]) and torch.equal(lse[i:i + n], lse[:n]) for i in range(0, n_seq * n, n))


def test_tree_of_single_tokens_is_the_decode(torch, ds4a):
    """One new token per sequence: the decode's result, its own row counted among the raw ones."""
    rng = np.random.default_rng(30)
    geom, first, parent, q, raw, comp = tree_case(rng, [1] * 5, [0, 9, 300, 77, 1500], 4, 16)
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    one = [(p, n + 1, r0, nc) for p, n, r0, nc in geom]
    want = paged.decode(shape_of(4), one, q, raw, comp)
    rows = [n for *_, n in geom]
    for par in (parent, None):
        got = run_tree(torch, ds4a, shape_of(4), geom, first, par, q, r, c)
        check_decode(*got, want, [n + 129 for n in rows])
    i32 = up(torch, np.array(one, dtype=np.int32))
    o, lse = ds4a.attn_decode_paged(shape_of(4), i32, up(torch, q), r, c, want_lse=True)
    check_decode(host(o), host(lse), want, [n + 129 for n in rows])


@pytest.mark.parametrize("chain", [False, True])
def test_tree_nan_in_a_query_stays_with_its_head(torch, ds4a, chain):
    rng = np.random.default_rng(32)
    geom, first, parent, q, raw, comp = tree_case(rng, [5, 6], [300, 20], 4, 16, chain=chain)
    want = step.attention(shape_of(4), geom, first, parent, q, raw, comp)
    q[4, 33, 100] = np.nan
    q[7, 0, 511] = np.inf
    o, lse = run_tree(torch, ds4a, shape_of(4), geom, first, parent, q, rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    assert np.isnan(o[4, 33]).all() and np.isnan(lse[4, 33])
    assert not np.isfinite(o[7, 0]).any() or np.isnan(o[7, 0]).all()
    o[4, 33], lse[4, 33], o[7, 0], lse[7, 0] = want[0][4, 33], want[1][4, 33], want[0][7, 0], want[1][7, 0]
    check_tree(o, lse, want)


# ------------------------------------------------------------------ the step as a whole

def same_pool(rows, seg):
    for name in ("k", "v"):
        assert np.array_equal(host(getattr(rows, name)).view(np.uint8), np.ascontiguousarray(seg[name]).view(np.uint8)), name
        if seg.get(name + "_scale") is not None:
            assert np.array_equal(host(getattr(rows, name + "_scale")), seg[name + "_scale"]), name


def write_rows(seg, slots, new, page):
    """New rows (fp16 [n, 512] for K and V) into the pool, as the append writes them."""
    for name, x in zip(("k",) if seg["v"] is seg["k"] else ("k", "v"), new):
        for s, row in zip(slots, x):
            if s < 0:
                continue
            if seg.get(name + "_scale") is not None:
                c, sc = fp8.quantize_rows(row[None])
                seg[name][s // page, s % page], seg[name + "_scale"][s // page, s % page] = c[0], sc[0]
            else:
                seg[name][s // page, s % page] = row


@pytest.mark.parametrize("recorded", [False, True])
@pytest.mark.parametrize("f8,shared,chain", [(False, True, False), (True, False, False), (False, False, True)])
def test_the_step_from_page_tables_to_page_tables(torch, ds4a, f8, shared, chain, recorded):
    """Several steps of one batch: pages for the new rows, the rows appended, attention, acceptance, the accepted rows
    moved, the pages of the others given back; as direct calls, and as two graphs that share the workspaces."""
    rng = np.random.default_rng(60 + f8 + 2 * chain)
    n, page, width, n_pages, ratio, window, T = 5, 16, 14, 60, 4, 64, 48
    shape = shape_of(ratio, window)
    comp_rows = [400, 3, 0, 77, 250]
    comp = make(rng, n, comp_rows, page, f8, shared)
    raw = make(rng, 1, [n_pages * page], page, f8, shared)  # a pool whose pages no sequence holds yet
    raw["table"] = np.full((n, width), -1, dtype=np.int32)
    c, r = rows_on(torch, ds4a, comp), rows_on(torch, ds4a, raw)
    free, n_free = rng.permutation(n_pages).astype(np.int32).tolist(), n_pages
    pos = np.array([x * ratio + 2 for x in comp_rows])
    raw0, n_raw = pos.copy(), np.zeros(n, dtype=int)
    prev = rng.integers(0, 2, n).astype(np.int32)

    stream = torch.cuda.Stream()
    zeros = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    d = dict(have=zeros(n), want=zeros(n), drop=zeros(n), slots=zeros(T), first=zeros(n + 1), short=zeros(1),
             geom=zeros(n, 4), parent=zeros(T), token=zeros(T), target=zeros(T), prev=up(torch, prev), path=zeros(n, T),
             count=zeros(n), next=zeros(n), have2=zeros(n), want2=zeros(n), first2=zeros(n + 1), short2=zeros(1),
             k=zeros(T, D, dtype=torch.float16), v=zeros(T, D, dtype=torch.float16),
             q=zeros(T, H, D, dtype=torch.float16), o=zeros(T, H, D, dtype=torch.float16), lse=zeros(T, H, dtype=torch.float32),
             free=up(torch, np.array(free, dtype=np.int32)), n_free=up(torch, np.array([n_free], dtype=np.int32)))
    wp = torch.empty(ds4a.page_tables_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    wt = torch.empty(ds4a.tree_paged_workspace_bytes(n, T), dtype=torch.uint8, device="cuda")
    par = None if chain else d["parent"]
    forward = [
        ds4a.prepare_page_tables(r.table, d["free"], d["n_free"], d["have"], d["want"], page, drop=d["drop"],
                                 slots=d["slots"], first=d["first"], n_short=d["short"], workspace=wp, stream=stream),
        ds4a.prepare_append_paged(r, d["k"], None if shared else d["v"], d["slots"], stream=stream),
        ds4a.prepare_tree_paged(shape, d["geom"], d["first"], d["q"], r, c, parent=par, workspace=wt, out=d["o"],
                                lse=d["lse"], stream=stream),
        ds4a.prepare_tree_accept(d["first"], d["token"], d["target"], parent=par, prev=d["prev"], path=d["path"],
                                 n_accepted=d["count"], next_token=d["next"], stream=stream),
        ds4a.prepare_commit_paged(r, d["geom"], d["path"], d["count"], stream=stream)]
    back = [ds4a.prepare_page_tables(r.table, d["free"], d["n_free"], d["have2"], d["want2"], page, slots=None,
                                     first=d["first2"], n_short=d["short2"], workspace=wp, stream=stream)]

    def run(calls):
        for f in calls:
            f()
    torch.cuda.synchronize()
    graphs = []
    if recorded:
        for calls in (forward, back):
            with ds4a.Graph(stream) as g:
                run(calls)
            graphs.append(g)
    accepted_some = accepted_none = 0
    for i in range(7):
        counts = rng.integers(0, 10, n)
        new = int(counts.sum())
        first = np.concatenate([[0], np.cumsum(counts)])
        drop = np.minimum(np.maximum(pos - window + 1 - raw0, 0), n_raw)
        gone = drop // page
        parent = None if chain else np.concatenate([tree_of(rng, m, False) for m in counts] + [np.zeros(T - new, int)])
        token, target = rng.integers(0, 2, T), rng.integers(0, 2, T)
        q, k, v = (rng.standard_normal(s).astype(np.float16) for s in ((T, H, D), (T, D), (T, D)))
        n_comp = np.array(comp_rows)
        # counted as after the dropped pages: the attention comes behind the page tables
        geom = np.stack([pos, n_raw - gone * page, raw0 + gone * page, n_comp], 1)
        for name, x in dict(have=n_raw, want=n_raw + counts, drop=drop, geom=geom, token=token, target=target,
                            have2=n_raw - gone * page + counts).items():
            d[name].copy_(up(torch, x.astype(np.int32)))
        if not chain:
            d["parent"].copy_(up(torch, parent.astype(np.int32)))
        for name, x in dict(q=q, k=k, v=v).items():
            d[name].copy_(up(torch, x))
        d["o"].fill_(7.0)
        torch.cuda.synchronize()
        graphs[0]() if recorded else run(forward)
        torch.cuda.synchronize()

        n_free, slots, first_, short = step.page_tables(raw["table"], free, n_free, n_raw, n_raw + counts, drop, page,
                                                        n_pages, T)
        assert np.array_equal(host(r.table), raw["table"]) and int(d["n_free"]) == n_free and int(d["short"]) == short == 0
        assert np.array_equal(host(d["slots"]), slots) and np.array_equal(host(d["first"]), first_)
        assert np.array_equal(first_, first)
        write_rows(raw, slots, (k, v), page)
        want = step.attention(shape, geom, first, parent, q, raw, comp)
        check_tree(host(d["o"])[:new], host(d["lse"])[:new], tuple(x[:new] for x in want))
        assert (host(d["o"])[new:] == 7).all()
        paths, nxt = step.accept(first, parent, token, target, host(d["prev"]), T)
        assert host(d["count"]).tolist() == [len(p) for p in paths] and host(d["next"]).tolist() == nxt
        step.commit(raw, geom, paths)
        same_pool(r, raw)

        taken = np.array([len(p) for p in paths])
        accepted_some += (taken > 1).sum()
        accepted_none += (taken == 0).sum()
        n_raw = n_raw - gone * page
        d["want2"].copy_(up(torch, (n_raw + taken).astype(np.int32)))
        torch.cuda.synchronize()
        graphs[1]() if recorded else run(back)
        torch.cuda.synchronize()
        n_free, *_ = step.page_tables(raw["table"], free, n_free, n_raw + counts, n_raw + taken, None, page, n_pages, 0)
        assert np.array_equal(host(r.table), raw["table"]) and int(d["n_free"]) == n_free
        assert np.array_equal(host(d["free"]), np.array(free, dtype=np.int32))
        pos, n_raw, raw0 = pos + taken, n_raw + taken, raw0 + gone * page
        d["prev"].copy_(d["next"])
    assert accepted_some and accepted_none
    assert n_pages == n_free + sum(-(-x // page) for x in n_raw)
    for g in graphs:
        g.close()


def test_the_documented_step_of_drafted_tokens(torch, ds4a):
    """The README's step, run as it stands: three steps of two sequences."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        (block,) = re.findall(r"```py\n(.*?)```", f.read(), re.S)
    rng = np.random.default_rng(71)
    n, page, n_pages, ratio = 2, 64, 9, 4
    comp = make(rng, n, [300, 40], page, False, True)
    raw = make(rng, 1, [n_pages * page], page, False, True)
    raw["table"] = np.full((n, 4), -1, dtype=np.int32)
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    free, n_free = rng.permutation(n_pages).astype(np.int32).tolist(), n_pages
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    geom = np.array([(1201, 0, 1201, 300), (163, 0, 163, 40)], dtype=np.int32)
    names = dict(torch=torch, ds4a=ds4a, geom=i32(geom), raw_table=r.table, raw=r, comp=c, free_pages=i32(free),
                 n_free=i32([n_free]), shape=shape_of(ratio), prev=i32([1, 0]))
    for counts in ([9, 70], [1, 5], [60, 60]):
        T = sum(counts)
        first = np.concatenate([[0], np.cumsum(counts)])
        parent = np.concatenate([tree_of(rng, m, False) for m in counts])
        token, target = rng.integers(0, 2, T), rng.integers(0, 2, T)
        q, k = rng.standard_normal((T, H, D)).astype(np.float16), rng.standard_normal((T, D)).astype(np.float16)
        names.update(first=i32(first), n_new=i32(counts), parent=i32(parent), token=i32(token), q=up(torch, q),
                     new_k=up(torch, k), choose=lambda o, t=target: i32(t))
        prev, have = host(names["prev"]), geom[:, 1].copy()
        exec(block, names)
        n_free, slots, *_ = step.page_tables(raw["table"], free, n_free, have, have + counts, None, page, n_pages, T)
        write_rows(raw, slots, (k,), page)
        want = step.attention(shape_of(ratio), geom, first, parent, q, raw, comp)
        check_tree(host(names["o"]), None, want)
        paths, nxt = step.accept(first, parent, token, target, prev, T)
        taken = np.array([len(p) for p in paths])
        step.commit(raw, geom, paths)
        same_pool(r, raw)
        n_free, *_ = step.page_tables(raw["table"], free, n_free, have + counts, have + taken, None, page, n_pages, 0)
        geom[:, :2] += taken[:, None].astype(np.int32)
        assert np.array_equal(host(names["geom"]), geom) and np.array_equal(host(r.table), raw["table"])
        assert int(names["n_free"]) == n_free and host(names["next_token"]).tolist() == nxt
        names["prev"] = names["next_token"]


@pytest.mark.parametrize("runs", [False, True])
def test_the_documented_step_on_a_layer_with_compressed_rows(torch, ds4a, runs):
    """The README's three blocks as they stand, until the windows have left their first pages and dozens of spans
    have ended: every node's result is that of decoding token by token along its path.  Or runs of drafts, as the text
    behind them says: the compressed rows of all their tokens first, and taken back to those of the accepted ones."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        before, block, behind = re.findall(r"```py(?:thon3)?\n(.*?)```", f.read(), re.S)
    rng = np.random.default_rng(72)
    if runs:
        before, roots = before.split("\nfor b in range(n_seq):")
        assert "append_compressed" in roots
    n, page, n_pages, ratio, start = 2, 64, 11, 4, [21, 8]
    shape = shape_of(ratio)
    pos = np.array(start)
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    comp = make(rng, n, [300, 300], page, False, True)
    comp["k"][:] = 0
    raw = make(rng, 1, [n_pages * page], page, False, True)
    raw["table"] = np.full((n, 4), -1, dtype=np.int32)
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    # What stands in the caches: positions from 0 on, in the state those of the span in progress.
    rows = [rng.standard_normal((int(x), D)).astype(np.float16) for x in pos]  # K = V of every position
    kvs, scores = ([rng.standard_normal((int(x), D)).astype(np.float32) for x in pos] for _ in range(2))
    geom = np.array([(x, x, 0, x // ratio) for x in pos], dtype=np.int32)
    free = rng.permutation(n_pages).tolist()
    for b in range(n):
        raw["table"][b, 0] = free.pop()
        raw["k"][raw["table"][b, 0], :pos[b]] = rows[b]
        pooled = compressor.pool(kvs[b][:pos[b] // ratio * ratio], scores[b][:pos[b] // ratio * ratio], ratio)
        comp["k"][comp["table"][b, 0], :len(pooled)] = pooled
    for seg, dev in ((raw, r), (comp, c)):
        dev.k.copy_(up(torch, seg["k"]))
    r.table.copy_(up(torch, raw["table"]))
    state = torch.zeros((2, n, ratio - 1, D), device="cuda")
    for b in range(n):
        for s, x in zip(state, (kvs, scores)):
            if pos[b] % ratio:
                s[b, :pos[b] % ratio] = up(torch, x[b][pos[b] // ratio * ratio:])
    names = dict(torch=torch, ds4a=ds4a, n_seq=n, geom=i32(geom), raw_table=r.table, raw=r, comp=c, comp_table=c.table,
                 free_pages=i32(free + [-1] * (n_pages - len(free))), n_free=i32([len(free)]), shape=shape,
                 prev=i32(rng.integers(0, 2, n)), state_kv=state[0], state_score=state[1],
                 n_state=[int(x) % ratio for x in pos])
    compared = 0
    for turn in range(200):
        # Trees of one root that end with the span: up to two more nodes in a generation.
        prev, parents, tokens, depths = host(names["prev"]), [], [], []
        for b in range(n):
            parent, depth = [-1], [0]
            for d in range(1, int(rng.integers(1, 10)) if runs else ratio - (int(pos[b]) + 1) % ratio):
                above = [t for t, x in enumerate(depth) if x == d - 1]
                for _ in range(1 if runs else int(rng.integers(1, 3))):
                    parent.append(int(rng.choice(above)))
                    depth.append(d)
            parents.append(parent)
            depths.append(depth)
            tokens.append([int(prev[b])] + rng.integers(0, 2, len(parent) - 1).tolist())
        counts = [len(x) for x in parents]
        T, first = sum(counts), np.concatenate([[0], np.cumsum(counts)])
        target = rng.integers(0, 2, T)
        q, k = rng.standard_normal((T, H, D)).astype(np.float16), rng.standard_normal((T, D)).astype(np.float16)
        kv, score = (rng.standard_normal((T, D)).astype(np.float32) for _ in range(2))
        names.update(first=i32(first), n_new=i32(counts), parent=None if runs else i32(np.concatenate(parents)),
                     q=up(torch, q), token=i32(np.concatenate(tokens)), new_k=up(torch, k), kv=up(torch, kv),
                     score=up(torch, score), choose=lambda o, t=target: i32(t))
        kept = (names["geom"][:, 3].clone(), state.clone(), list(names["n_state"]))
        exec(before, names)
        if runs:
            for b in range(n):
                names["append_compressed"](b, torch.arange(first[b], first[b + 1], device="cuda"))
        exec(block, names)
        path, taken = host(names["path"]), host(names["n_accepted"])
        paths, nxt = step.accept(first, np.concatenate(parents), np.concatenate(tokens), target, prev, 128)
        assert [path[b, :taken[b]].tolist() for b in range(n)] == paths and (taken >= 1).all()
        assert host(names["next_token"]).tolist() == nxt and int(names["n_short"]) == 0
        if turn % 8 == 0 or turn > 190:
            cache, c_table = host(c.k), host(c.table)
            for b in range(n):
                ways = []
                for t, u in enumerate(parents[b]):
                    ways.append((ways[u] if u >= 0 else []) + [t])
                    at = first[b] + t
                    seq_rows = np.concatenate([rows[b], k[first[b] + np.array(ways[t])]])
                    p, ended = len(seq_rows) - 1, len(seq_rows) // ratio
                    pooled = cache[c_table[b, np.arange(ended) // page], np.arange(ended) % page]
                    segs = []
                    for x in (seq_rows, pooled):
                        x = np.concatenate([x, np.zeros((-len(x) % page, D), dtype=np.float16)]).reshape(-1, page, D)
                        segs.append(dict(k=x, v=x, table=np.arange(len(x), dtype=np.int32)[None]))
                    want = paged.decode(shape, [(p, len(seq_rows), 0, ended)], q[at:at + 1], *segs)
                    check_decode(host(names["o"])[at:at + 1], None, want, [min(128, p + 1) + ended])
                    compared += 1
        if runs:
            names["geom"][:, 3], names["n_state"] = kept[0], kept[2]
            state.copy_(kept[1])
            for b in range(n):
                names["append_compressed"](b, (names["first"][b] + names["path"][b, :taken[b]]).long())
        else:
            exec(behind, names)
        for b in range(n):
            took = first[b] + np.array(paths[b])
            rows[b], kvs[b], scores[b] = (np.concatenate([x, y[took]]) for x, y in
                                          ((rows[b], k), (kvs[b], kv), (scores[b], score)))
        pos = pos + taken
        g = host(names["geom"])
        assert g[:, 0].tolist() == pos.tolist() and (g[:, 1] + g[:, 2] == pos).all() and (g[:, 3] == pos // ratio).all()
        names["prev"] = names["next_token"]
    assert compared > 100 and (host(names["geom"])[:, 2] >= page).all()
    assert int(names["n_free"]) == n_pages - sum(-(-int(x) // page) for x in host(names["geom"])[:, 1])
    # The compressed rows, by the compressor's definition.  (Weights from scores up to 10 apart: an exponent is off by
    # 10 log2(e) 2^-24, a weight and a quotient by another 2^-22 each: under 2^-18 of the span's largest row; then fp16.)
    for b in range(n):
        ended = pos[b] // ratio
        got = host(c.k)[c_table[b, np.arange(ended) // page], np.arange(ended) % page].astype(np.float64)
        most = np.abs(kvs[b][:ended * ratio]).reshape(ended, ratio, D).max(1)
        want = compressor.pool(kvs[b][:ended * ratio], scores[b][:ended * ratio], ratio)
        assert (np.abs(got - want) <= F16 * np.abs(want) + 2.0 ** -18 * most + 2.0 ** -25).all()


def test_steps_on_two_streams_at_once(torch, ds4a):
    """Attention, acceptance and commits in flight on two streams, outputs and workspaces made by the calls: a job's
    results are the same bits every time."""
    rng = np.random.default_rng(70)
    jobs = []
    for k in range(2):
        geom, first, parent, q, raw, comp = tree_case(rng, [9 + k, 30, 2], [2000, 700 + k, 5], 4, 16, bool(k), True)
        i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
        token, target = rng.integers(0, 2, len(q)), rng.integers(0, 2, len(q))
        jobs.append(dict(geom=i32(geom), first=i32(first), parent=i32(parent), q=up(torch, q), raw=rows_on(torch, ds4a, raw),
                         comp=rows_on(torch, ds4a, comp), token=i32(token), target=i32(target), stream=torch.cuda.Stream(),
                         want=step.attention(shape_of(4), geom, first, parent, q, raw, comp),
                         paths=step.accept(first, parent, token, target, None, len(q))))
    torch.cuda.synchronize()
    outs = []
    for _ in range(12):
        for j in jobs:
            o, lse = ds4a.attn_tree_paged(shape_of(4), j["geom"], j["first"], j["q"], j["raw"], j["comp"],
                                          parent=j["parent"], want_lse=True, stream=j["stream"])
            outs.append((o, lse, *ds4a.tree_accept(j["first"], j["token"], j["target"], parent=j["parent"],
                                                   stream=j["stream"])))
    torch.cuda.synchronize()
    for k, j in enumerate(jobs):
        check_tree(host(outs[k][0]), host(outs[k][1]), j["want"])
        assert host(outs[k][3]).tolist() == [len(p) for p in j["paths"][0]] and host(outs[k][4]).tolist() == j["paths"][1]
        for again in outs[k + 2::2]:
            assert all(torch.equal(a, b) for a, b in zip(again, outs[k]))


def test_all_calls_of_the_step_on_two_streams_at_once(torch, ds4a):
    """Page tables, attention, acceptance and commits in flight on two streams, each job with pools, tables and lists
    of its own, outputs and workspaces made by the calls: every round's results, and what all rounds leave behind."""
    rng = np.random.default_rng(73)
    i32 = lambda a: up(torch, np.asarray(a, dtype=np.int32))  # noqa: E731
    rounds, jobs = 8, []
    for k in range(2):
        counts = [9 + k, 30, 2]
        geom, first, parent, q, raw, comp = tree_case(rng, counts, [600, 300 + k, 5], 4, 16, bool(k), True)
        if k:
            raw["k_scale"][np.isnan(raw["k_scale"])] = 3.0  # (to be compared; of rows that nobody sees)
        token, target = rng.integers(0, 2, len(q)), rng.integers(0, 2, len(q))
        prev = token[first[:-1]]
        have, want, _, table, free, n_free, n_pages = page_case(rng, 40 + k, 16, 90, 60, False, 150)
        jobs.append(dict(
            host=dict(geom=geom, first=first, parent=parent, q=q, raw=raw, comp=comp, have=have, want=want, table=table,
                      free=free.tolist(), n_free=n_free, n_pages=n_pages, slots=int(np.maximum(want - have, 0).sum()),
                      paths=step.accept(first, parent, token, target, prev, 128)),
            geom=i32(geom), first=i32(first), parent=i32(parent), q=up(torch, q), raw=rows_on(torch, ds4a, raw),
            comp=rows_on(torch, ds4a, comp), token=i32(token), target=i32(target), prev=i32(prev), have=i32(have),
            want=i32(want), table=i32(table), free=i32(free), n_free=i32([n_free]), stream=torch.cuda.Stream()))
    assert any(len(p) > 2 for j in jobs for p in j["host"]["paths"][0])
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(rounds):
        for j, out in zip(jobs, outs):
            s, h = j["stream"], j["host"]
            there = ds4a.page_tables(j["table"], j["free"], j["n_free"], j["have"], j["want"], 16, n_slots=h["slots"],
                                     stream=s)
            o = ds4a.attn_tree_paged(shape_of(4), j["geom"], j["first"], j["q"], j["raw"], j["comp"], parent=j["parent"],
                                     stream=s)
            taken = ds4a.tree_accept(j["first"], j["token"], j["target"], parent=j["parent"], prev=j["prev"], stream=s)
            ds4a.commit_paged(j["raw"], j["geom"], taken[0], taken[1], stream=s)
            ds4a.page_tables(j["table"], j["free"], j["n_free"], j["want"], j["have"], 16, stream=s)
            out.append((there, o, taken))
    torch.cuda.synchronize()
    for j, out in zip(jobs, outs):
        h = j["host"]
        for i, (there, o, taken) in enumerate(out):
            h["n_free"], slots, first, short = step.page_tables(h["table"], h["free"], h["n_free"], h["have"], h["want"], None,
                                                                16, h["n_pages"], h["slots"])
            assert np.array_equal(host(there[0]), slots) and np.array_equal(host(there[1]), first) and int(there[2]) == short
            if i in (0, rounds - 1):
                want = step.attention(shape_of(4), h["geom"], h["first"], h["parent"], h["q"], h["raw"], h["comp"])
                check_tree(host(o), None, want)
            paths, nxt = h["paths"]
            assert [p[:n] for p, n in zip(host(taken[0]).tolist(), host(taken[1]).tolist())] == paths
            assert (host(taken[0]) >= 0).sum() == sum(map(len, paths)) and host(taken[2]).tolist() == nxt
            step.commit(h["raw"], h["geom"], paths)
            h["n_free"], *_ = step.page_tables(h["table"], h["free"], h["n_free"], h["want"], h["have"], None, 16, h["n_pages"], 0)
        same_pool(j["raw"], h["raw"])
        assert np.array_equal(host(j["table"]), h["table"]) and np.array_equal(host(j["free"]), h["free"])
        assert int(j["n_free"]) == h["n_free"]


def test_step_calls_of_empty_batches(torch, ds4a):
    """No sequence, or no new token: nothing is written, and nothing fails."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = ds4a.PagedRows(torch.zeros((4, 16, D), dtype=torch.float16, device="cuda"), None, i32(2, 3))
    o = ds4a.attn_tree_paged(shape_of(4), i32(2, 4), i32(3), torch.zeros((0, H, D), dtype=torch.float16, device="cuda"), rows)
    assert o.shape == (0, H, D)
    none = ds4a.PagedRows(rows.k, None, i32(0, 3))
    q = torch.zeros((3, H, D), dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 5)
    ds4a.attn_tree_paged(shape_of(4), i32(0, 4), i32(1), q, none, out=out)
    assert (out == 5).all()
    path, count, nxt = ds4a.tree_accept(i32(3), i32(0), i32(0), width=4)
    assert (path == -1).all() and count.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
    assert ds4a.tree_accept(i32(1), i32(0), i32(0), width=4)[0].shape == (0, 4)
    ds4a.commit_paged(rows, i32(2, 4), i32(2, 0), i32(2))
    ds4a.commit_paged(none, i32(0, 4), i32(0, 4), i32(0))
    slots, first, short = ds4a.page_tables(i32(0, 3), i32(4), i32(1), i32(0), i32(0), 16, n_slots=3)
    assert slots.tolist() == [-1] * 3 and first.tolist() == [0] and short.tolist() == [0]
    torch.cuda.synchronize()
