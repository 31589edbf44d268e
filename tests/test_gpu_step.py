"""A step with several new tokens per sequence against the fp64 oracle (needs a GB300).

Page tables, accepted paths and moved rows are whole numbers and copies: bit for bit.
"""

import numpy as np
import pytest

from oracle import paged, step
from test_gpu_paged import device_error_word_stays_clear, ds4a, host, rows_on, torch, up  # noqa: F401
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
    (1024, 16, 90, 40, 2000), (1025, 8, 30, 20, 100), (2500, 24, 60, 100, 20000), (2, 128, 5000, 9000, 200)])
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
