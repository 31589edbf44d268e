"""Refusals of the calls of a step with several new tokens, without a GPU, and
the step's oracle by hand."""

import ctypes
import math

import numpy as np
import pytest
import torch

from mqa_flash_attention_gb300 import ds4a
from oracle import paged, step
from test_paged_checks import AT, I32, SHAPE, elsewhere, lib, needs_no_gpu, passes, raises, seg  # noqa: F401


def lists(**kw):
    base = dict(table=AT, table_stride=32, max_pages=8, page_rows=16, n_pages=100, free_pages=2 * AT, n_free=3 * AT,
                have=4 * AT, want=5 * AT, drop=None, slots=6 * AT, n_slots=50, first=7 * AT, n_short=8 * AT)
    base.update(kw)
    return ds4a.PageLists(*[base[n] for n, _ in ds4a.PageLists._fields_])


def pages(lib, n=3, ws=1 << 30, nbytes=1 << 20, **kw):
    return elsewhere(lib.ds4a_page_tables, n, ctypes.byref(lists(**kw)), ws, nbytes, None)


@needs_no_gpu
def test_page_tables_arguments_are_checked(lib):
    assert passes(pages(lib)) and passes(pages(lib, drop=9 * AT)) and passes(pages(lib, slots=None, n_slots=0))
    assert passes(pages(lib, want=4 * AT, drop=4 * AT))
    assert pages(lib, n=0) == ds4a.OK
    for bad in (dict(n=-1), dict(n=(1 << 20) + 1), dict(table=None), dict(table=AT + 2), dict(table_stride=28),
                dict(table_stride=34), dict(max_pages=0), dict(page_rows=0), dict(n_pages=0), dict(n_slots=-1),
                dict(max_pages=1 << 10, table_stride=1 << 12, page_rows=(1 << 20) + 1, n_pages=1),
                dict(page_rows=1 << 16, n_pages=1 << 15), dict(free_pages=None), dict(n_free=None), dict(have=None),
                dict(want=None), dict(first=None), dict(n_short=None), dict(slots=None), dict(have=AT * 4 + 1),
                dict(drop=AT * 9 + 2), dict(slots=6 * AT + 1), dict(first=7 * AT + 3),
                # ranges that overlap
                dict(have=AT + 64), dict(slots=5 * AT + 8), dict(free_pages=6 * AT + 196), dict(n_free=2 * AT + 396),
                dict(n_short=7 * AT + 12), dict(first=AT + 92), dict(drop=8 * AT)):
        assert pages(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    need = lib.ds4a_page_tables_workspace_size(3)
    assert need > 0 and lib.ds4a_page_tables_workspace_size(0) == 0
    for bad in (dict(ws=None), dict(ws=AT + 64), dict(nbytes=need - 1)):
        assert pages(lib, **bad) == ds4a.ERR_WORKSPACE, bad


@needs_no_gpu
def test_page_tables_workspace_apart_from_the_lists(lib):
    need = lib.ds4a_page_tables_workspace_size(3)
    base = lists(drop=9 * AT)
    sizes = dict(table=2 * 32 + 32, free_pages=400, n_free=4, have=12, want=12, drop=12, slots=200, first=16, n_short=4)
    for name, size in sizes.items():
        at = getattr(base, name)
        assert pages(lib, drop=9 * AT, ws=at) == ds4a.ERR_INVALID_ARG, name
        assert passes(pages(lib, drop=9 * AT, ws=at + (size + 255) // 256 * 256)), name
        assert passes(pages(lib, drop=9 * AT, ws=at - 256)), name  # (64 bytes are used)
        assert pages(lib, **dict(dict(drop=9 * AT), **{name: (1 << 30) + need - 4})) == ds4a.ERR_INVALID_ARG, name
        assert passes(pages(lib, **dict(dict(drop=9 * AT), **{name: (1 << 30) + need}))), name


def accept(lib, n=3, n_tok=20, first=AT, parent=2 * AT, token=3 * AT, target=4 * AT, prev=5 * AT, path=6 * AT, stride=40,
           width=10, count=7 * AT, nxt=8 * AT):
    return elsewhere(lib.ds4a_tree_accept, n, n_tok, first, parent, token, target, prev, path, stride, width, count, nxt,
                     None)


@needs_no_gpu
def test_accept_arguments_are_checked(lib):
    assert passes(accept(lib)) and passes(accept(lib, parent=None, prev=None))
    assert passes(accept(lib, width=0, path=None, stride=0)) and passes(accept(lib, n_tok=0, token=None, target=None))
    assert passes(accept(lib, token=4 * AT))
    assert accept(lib, n=0) == ds4a.OK
    for bad in (dict(n=-1), dict(n_tok=-1), dict(width=-1), dict(first=None), dict(first=AT + 2), dict(token=None),
                dict(target=None), dict(parent=AT * 2 + 1), dict(token=AT * 3 + 2), dict(prev=5 * AT + 2),
                dict(path=None), dict(path=6 * AT + 2), dict(stride=36), dict(stride=42), dict(count=None), dict(nxt=None),
                dict(count=7 * AT + 1), dict(path=2 * AT + 76), dict(count=AT + 12), dict(nxt=7 * AT + 8),
                dict(nxt=5 * AT), dict(count=6 * AT + 116), dict(n=(1 << 20) + 1)):
        assert accept(lib, **bad) == ds4a.ERR_INVALID_ARG, bad


def commit(lib, rows=None, n=3, geom=5 * AT, path=6 * AT, stride=40, width=10, count=7 * AT):
    return elsewhere(lib.ds4a_commit_paged, n, ctypes.byref(rows or seg()), geom, path, stride, width, count, None)


@needs_no_gpu
def test_commit_arguments_are_checked(lib):
    assert passes(commit(lib)) and passes(commit(lib, seg(v=AT)))
    f8 = dict(row_stride=512, page_stride=8192)
    assert passes(commit(lib, seg(k_scale=11 * AT, v_scale=12 * AT, **f8)))
    assert commit(lib, n=0) == ds4a.OK and commit(lib, width=0, path=None) == ds4a.OK
    for bad in (dict(n=-1), dict(width=-1), dict(geom=None), dict(geom=AT + 4), dict(path=None), dict(path=AT + 1),
                dict(stride=36), dict(stride=41), dict(count=None), dict(count=AT + 2), dict(rows=seg(max_pages=0)),
                dict(rows=seg(table=None)), dict(rows=seg(v=None)), dict(rows=seg(k=AT + 8)), dict(n=(1 << 20) + 1),
                dict(rows=seg(k_scale=11 * AT, v_scale=11 * AT, **f8))):
        assert commit(lib, **bad) == ds4a.ERR_INVALID_ARG, bad


def tree(lib, n=3, n_tok=20, shape=None, geom=5 * AT, ws=1 << 30, nbytes=None, **kw):
    base = dict(q=1 << 35, q_tok_stride=65536, first=6 * AT, parent=7 * AT, raw=seg(), comp=seg(), o=1 << 36,
                o_tok_stride=65536, lse=1 << 37)
    base.update(kw)
    X = ds4a.PagedTree(*[base[n] for n, _ in ds4a.PagedTree._fields_])
    S = ds4a.make_layout(dict(SHAPE, **(shape or {})))
    if shape and "ratio" in shape:
        S.ratio = shape["ratio"]
    need = lib.ds4a_attn_tree_paged_workspace_size(n, n_tok)
    return elsewhere(lib.ds4a_attn_tree_paged, n, n_tok, ctypes.byref(S), geom, ctypes.byref(X), ws,
                     need if nbytes is None else nbytes, None)


@needs_no_gpu
def test_tree_arguments_are_checked(lib):
    f8 = dict(row_stride=512, page_stride=8192, k_scale=AT, v_scale=AT)
    none = seg(max_pages=0, k=None)
    assert passes(tree(lib)) and passes(tree(lib, parent=None, lse=None)) and passes(tree(lib, raw=none))
    assert passes(tree(lib, comp=none)) and passes(tree(lib, raw=seg(**f8), comp=seg(**f8)))
    assert passes(tree(lib, raw=none, comp=none)) and passes(tree(lib, comp=seg(page_rows=1, page_stride=1024)))
    assert tree(lib, n=0) == ds4a.OK and tree(lib, n_tok=0) == ds4a.OK
    big = dict(page_rows=1 << 27, n_pages=8, page_stride=1 << 37, table_stride=32, max_pages=8)
    for bad in (dict(n=-1), dict(n_tok=-1), dict(n=(1 << 20) + 1), dict(n_tok=(1 << 20) + 1), dict(q=None), dict(q=AT + 8),
                dict(q_tok_stride=65520), dict(q_tok_stride=65544), dict(o=None), dict(o=AT + 4), dict(o_tok_stride=0),
                dict(lse=AT + 2), dict(first=None), dict(first=AT + 1), dict(parent=AT + 2), dict(geom=None),
                dict(geom=AT + 8), dict(shape=dict(window=0)), dict(shape=dict(ratio=0)), dict(shape=dict(scale=math.inf)),
                dict(shape=dict(scale=math.nan)), dict(shape=dict(scale=3e38)), dict(comp=seg(**f8)), dict(raw=seg(k=None)),
                dict(comp=seg(v=None)), dict(raw=seg(page_rows=0)), dict(comp=seg(table=None)), dict(raw=seg(max_pages=-1)),
                dict(raw=seg(**big), comp=seg()),
                # ranges that overlap
                dict(o=(1 << 35) + 65536), dict(o=(1 << 35) - 19 * 65536), dict(lse=(1 << 36) + 16), dict(lse=7 * AT + 76),
                dict(lse=6 * AT - 5116), dict(o=5 * AT), dict(ws=1 << 35), dict(ws=(1 << 36) - 256), dict(lse=1 << 30)):
        assert tree(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    need = lib.ds4a_attn_tree_paged_workspace_size(3, 20)
    assert need > 0 and lib.ds4a_attn_tree_paged_workspace_size(0, 5) == 0
    for bad in (dict(ws=None), dict(ws=(1 << 30) + 128), dict(nbytes=need - 1)):
        assert tree(lib, **bad) == ds4a.ERR_WORKSPACE, bad


@needs_no_gpu
def test_tree_outputs_apart_from_the_rows(lib):
    """o, lse and the workspace against pools, scales and tables of both segments; a segment without rows has none."""
    need = lib.ds4a_attn_tree_paged_workspace_size(3, 20)
    far = {n: (72 + i) << 30 for i, n in enumerate(("k", "v", "k_scale", "v_scale", "table"))}
    for which in ("raw", "comp"):
        for f8 in (False, True):
            row = 512 if f8 else 1024
            kw = dict(far, row_stride=row, page_stride=16 * row)
            if not f8:
                kw.update(k_scale=None, v_scale=None)
            other = dict(raw=seg(max_pages=0, k=None), comp=seg(max_pages=0, k=None))
            rows = dict(other, **{which: seg(**kw)})
            assert passes(tree(lib, **rows))
            ends = dict(k=8 * 16 * row, v=8 * 16 * row, k_scale=8 * 64, v_scale=8 * 64, table=2 * 32 + 32)
            for name, size in ends.items():
                if kw[name] is None:
                    continue
                at = kw[name]
                for bad in (dict(o=at + size - 16), dict(o=at - 20 * 65536 + 16), dict(lse=at + size - 4),
                            dict(lse=at - 20 * 256 + 4), dict(ws=at), dict(ws=at - (need - 1) // 256 * 256)):
                    assert tree(lib, **rows, **bad) == ds4a.ERR_INVALID_ARG, (which, name, bad)
                for good in (dict(o=at + (size + 15) // 16 * 16), dict(o=at - 20 * 65536), dict(lse=at + size),
                             dict(lse=at - 20 * 256), dict(ws=at + (size + 255) // 256 * 256)):
                    assert passes(tree(lib, **rows, **good)), (which, name, good)
            if which == "raw":
                empty = dict(raw=seg(max_pages=0, **{k: v for k, v in kw.items()}), comp=other["comp"])
                assert passes(tree(lib, **empty, o=far["k"], lse=far["v"]))


# ------------------------------------------------------------------ binding

def i32(*shape):
    return torch.zeros(shape, dtype=I32)


def test_step_calls_refuse_what_does_not_fit():
    """Sizes, types and strides, and then that host tensors are no device tensors."""
    good = dict(table=i32(3, 8), free_pages=i32(100), n_free=i32(1), have=i32(3), want=i32(3), page_rows=16,
                slots=i32(9), first=i32(4), n_short=i32(1), workspace=torch.zeros(256, dtype=torch.uint8))
    raises("CUDA tensor", ds4a.prepare_page_tables, **good)
    for bad, match in ((dict(table=i32(2, 8)), "table"), (dict(table=i32(3)), "table"),
                       (dict(table=torch.zeros(3, 8)), "table"), (dict(table=i32(8, 3).T), "table"),
                       (dict(table=i32(1, 8).expand(3, 8)), "table")):
        raises(match, ds4a.prepare_page_tables, **dict(good, **bad))
    good = dict(first=i32(4), token=i32(20), target=i32(20), path=i32(3, 5), n_accepted=i32(3), next_token=i32(3))
    for bad, match in ((dict(path=i32(2, 5)), "path"), (dict(path=None), "path"), (dict(path=i32(1, 5).expand(3, 5)), "path"),
                       (dict(path=torch.zeros(3, 5)), "path"), (dict(first=i32(0)), "first")):
        raises(match, ds4a.prepare_tree_accept, **dict(good, **bad))


def test_tree_refuses_what_does_not_fit(monkeypatch):
    def f16(*shape):
        return torch.zeros(shape, dtype=torch.float16)
    rows = ds4a.PagedRows(f16(4, 16, 512), None, i32(2, 3))
    good = dict(shape=SHAPE, seq_geom=i32(2, 4), first=i32(3), q=f16(9, 64, 512), raw=rows, out=f16(9, 64, 512),
                workspace=torch.zeros(1, dtype=torch.uint8))
    raises("CUDA tensor", ds4a.prepare_tree_paged, **good)
    monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
    for bad, match in ((dict(q=f16(9, 64, 256)), "q must"), (dict(out=f16(8, 64, 512)), "out"), (dict(first=i32(2)), "first"),
                       (dict(out=f16(1, 64, 512).expand(9, 64, 512)), "out"), (dict(parent=i32(8)), "parent"),
                       (dict(parent=torch.zeros(9)), "parent"), (dict(lse=torch.zeros(9, 63)), "lse"),
                       (dict(seq_geom=i32(2, 3)), "seq_geom"), (dict(raw=ds4a.PagedRows(f16(4, 16, 512))), "page table"),
                       (dict(comp=ds4a.PagedRows(f16(4, 16, 512), None, i32(1, 3))), "comp.table")):
        raises(match, ds4a.prepare_tree_paged, **dict(good, **bad))


@pytest.mark.parametrize("name,bad", [("have", i32(2)), ("have", i32(6)[::2]), ("want", torch.zeros(3)),
                                      ("first", i32(3)), ("n_short", i32(0)), ("drop", i32(2)), ("n_free", i32(1, 1))])
def test_whole_numbers_of_the_wrong_kind_are_refused(name, bad, monkeypatch):
    monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
    good = dict(table=i32(3, 8), free_pages=i32(100), n_free=i32(1), have=i32(3), want=i32(3), page_rows=16,
                slots=i32(9), first=i32(4), n_short=i32(1), workspace=torch.zeros(256, dtype=torch.uint8))
    if name == "have" and bad.shape[0] == 2:
        good["table"] = i32(1, 8)
        name, match = "have", "table"
    else:
        match = name
    raises(match, ds4a.prepare_page_tables, **dict(good, **{name: bad}))


@pytest.mark.parametrize("n,tree,width,cols", [(5, True, None, 5), (32768, True, None, 128), (32768, False, None, 32768),
                                               (32768, True, 64, 64), (32768, False, 7, 7), (0, True, None, 0)])
def test_accept_makes_a_path_as_wide_as_a_tree(monkeypatch, n, tree, width, cols):
    """Not of all sequences' nodes: 512 trees of 64 would write 64 MB."""
    made = []
    monkeypatch.setattr(ds4a, "prepare_tree_accept", lambda *a, path, **kw: made.append(path) or (lambda: None))
    path, count, _ = ds4a.tree_accept(i32(513), i32(n), i32(n), parent=i32(n) if tree else None, width=width)
    assert made[0] is path and path.shape == (512, cols) and count.shape == (512,)


# ------------------------------------------------------------------ the oracle by hand

def test_page_tables_by_hand():
    """Sequence 0 drops its first page and grows over a page's end; 1 gives a page back; 2 finds the list empty."""
    table = np.array([[3, 1, -1], [0, 5, -1], [-1, -1, -1]], dtype=np.int32)
    free = [4, -1, -1, -1, -1, -1]
    n_free, slots, first, short = step.page_tables(table, free, 1, [7, 6, 0], [10, 3, 9], [5, 0, 0], 4, 6, 14)
    # given back: 3, then 5 -> list 4 3 5; taken: 5 (sequence 0), then 3, 4 and none (sequence 2)
    assert table.tolist() == [[1, 5, -1], [0, -1, -1], [3, 4, -1]]
    assert n_free == 0 and short == 1 and first.tolist() == [0, 3, 3, 12]
    assert slots.tolist() == [1 * 4 + 3, 5 * 4, 5 * 4 + 1] + [12, 13, 14, 15, 16, 17, 18, 19, -1] + [-1, -1]


def test_accept_by_hand():
    #      0 -> 1, 2;  1 -> 3;  2 -> 4, 5
    parent = np.array([-1, 0, 0, 1, 2, 2])
    token = np.array([7, 8, 9, 1, 2, 3])
    target = np.array([9, 1, 3, 0, 0, 6])
    assert step.accept([0, 6], parent, token, target, [7], 9) == ([[0, 2, 5]], [6])
    assert step.accept([0, 6], parent, token, target, [6], 9) == ([[]], [6])
    assert step.accept([0, 6], parent, token, target, None, 2) == ([[0, 2]], [3])
    assert step.accept([0, 0], parent, token, target, None, 2) == ([[]], [-1])


def test_seen_by_hand():
    """A tree of four at position 6, rows 4 and 5 cached, window 3."""
    shape = dict(window=3, ratio=2, scale=1.0)
    got = step.seen(shape, (6, 2, 4, 9), np.array([-1, 0, 0, 2]), 0, 4, 100, 100)
    assert got == [([0, 1, 2], [0, 1, 2]), ([1, 2, 3], [0, 1, 2, 3]), ([1, 2, 4], [0, 1, 2, 3]), ([2, 4, 5], [0, 1, 2, 3])]


def whole_history(rng, n_rows, n_spans):
    """Rows of one sequence from position 0 on, in pages, and its compressed rows."""
    def rows(n):
        k = rng.standard_normal((-(-n // 8), 8, 512)).astype(np.float16)
        return dict(k=k, v=k, table=np.arange(len(k), dtype=np.int32)[None])
    return rows(n_rows), rows(n_spans)


def decoded(shape, raw, comp, q, p, path, n_raw):
    """Token-by-token decode at position p: the cached rows 0 .. n_raw - 1, then those of ``path``, and every
    compressed row whose span has ended."""
    at = list(range(n_raw)) + [n_raw + t for t in path]
    k = raw["k"].reshape(-1, 512)[at]
    k = np.concatenate([k, np.zeros((-len(k) % 8, 512), dtype=np.float16)]).reshape(-1, 8, 512)
    own = dict(k=k, v=k, table=np.arange(len(k), dtype=np.int32)[None])
    o, lse, *_ = paged.decode(shape, [(p, len(at), 0, 1 << 20)], q[None], own, comp)
    return o[0], lse[0]


@pytest.mark.parametrize("ratio,pos", [(4, 11), (4, 12), (2, 9), (16, 40)])
def test_a_run_is_decode_token_by_token(ratio, pos):
    """With the compressed rows of its own tokens in the cache and counted."""
    rng = np.random.default_rng(ratio)
    n, shape = 13, dict(ratio=ratio, window=9, scale=1 / math.sqrt(512))
    raw, comp = whole_history(rng, pos + n, (pos + n) // ratio)
    q = rng.standard_normal((n, 64, 512)).astype(np.float16)
    o, lse, *_ = step.attention(shape, [(pos, pos, 0, (pos + n) // ratio)], [0, n], None, q, raw, comp)
    for t in range(n):
        want = decoded(shape, raw, comp, q[t], pos + t, range(t + 1), pos)
        assert np.allclose(o[t], want[0], rtol=0, atol=1e-12) and np.allclose(lse[t], want[1], rtol=0, atol=1e-12)


@pytest.mark.parametrize("pos", [8, 9, 10, 11])
def test_a_tree_is_decode_until_a_span_ends_on_a_branch(pos):
    """A root, two branches of three: equal to decode along each node's path while n_comp counts the spans that
    have ended on it (the root's row may have been appended), and short of the branch's compressed row behind that."""
    rng = np.random.default_rng(pos)
    ratio, parent = 4, np.array([-1, 0, 0, 1, 2, 3, 4])
    paths = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [0, 1, 3, 5], [0, 2, 4, 6]]
    shape = dict(ratio=ratio, window=128, scale=1 / math.sqrt(512))
    raw, comp = whole_history(rng, pos + 7, 8)  # (branches' rows differ: those of one of them)
    n_comp = (pos + 1) // ratio                 # the root's among them
    q = rng.standard_normal((7, 64, 512)).astype(np.float16)
    o, lse, *_ = step.attention(shape, [(pos, pos, 0, n_comp)], [0, 7], parent, q, raw, comp)
    same = 0
    for t, path in enumerate(paths):
        p = pos + len(path) - 1
        want = decoded(shape, raw, comp, q[t], p, path, pos)
        equal = np.allclose(o[t], want[0], rtol=0, atol=1e-12) and np.allclose(lse[t], want[1], rtol=0, atol=1e-12)
        assert equal == ((p + 1) // ratio <= n_comp)
        same += equal
    assert same == {8: 5, 9: 3, 10: 1, 11: 7}[pos]


def test_the_header_names_a_tree_s_tokens():
    import os
    import re
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "ds4a.h")) as f:
        assert re.search(r"#define DS4A_TREE_TOKENS (\d+)", f.read()).group(1) == str(ds4a.TREE_TOKENS)
