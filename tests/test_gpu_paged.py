"""The paged cache operators and the norm against the fp64 oracle (needs a GB300).

Tolerances, from the arithmetic (a rounding to fp16 is off by at most 2^-11 of
the value, one to fp32 by 2^-24):

* decode: the weights are rounded once to fp16 for the product (2^-11 of each
  term) and the output is rounded (2^-11): twice 2^-11 of A = sum_j w_j |v_j|,
  and a tenth for fp32 arithmetic and products of these.  A score is a sum of 512 fp32 products: off by at most
  e = 512 * 2^-23 * scale * sum |q||k| (2^-23 covers truncating adders), which
  moves a weight by a factor of at most exp(2 e).  fp16 numbers below 2^-14
  have a fixed step: 2^-25.
* log-sum-exp: e, and fp32 sums of N weights, exp2 and log: (N / 128 + 40) * 2^-23.
* received weights: a factor exp(e), exponents of size |s| + |lse| held to
  2^-23, and 64 additions.
* norm: at most 40 fp32 roundings (2^-18) before the one that is asserted; an
  E4M3 code is within half a step of the exact quotient, which those roundings
  may carry across a tie.
* whole numbers, moved rows, appended rows, residual sums: bit for bit.
"""

import os
import re

import numpy as np
import pytest

from oracle import fp8, paged
from test_paged_oracle import make

pytestmark = pytest.mark.gpu

H, D = 64, 512
F16 = 2.0 ** -11


@pytest.fixture(scope="module")
def torch():
    import torch as _torch
    from mqa_flash_attention_gb300 import build
    build.build()
    assert _torch.cuda.is_available()
    return _torch


@pytest.fixture(scope="module")
def ds4a(torch):
    from mqa_flash_attention_gb300 import ds4a as _ds4a
    _ds4a.lib()
    return _ds4a


@pytest.fixture(autouse=True)
def device_error_word_stays_clear(ds4a):
    ds4a.device_error_word(clear=True)
    yield
    w = ds4a.device_error_word(clear=True)
    assert w == 0, f"a device wait ran out during this test: error word {w:#010x}"


def up(torch, a):
    return None if a is None else torch.from_numpy(np.array(a, order="C", copy=True)).cuda()


def host(t):
    return t.detach().cpu().numpy()


def shape_of(ratio=4, window=128, scale=1.0 / np.sqrt(512.0)):
    return dict(T=1, q_pos0=0, n_raw=0, raw_pos0=0, n_comp=0, ratio=ratio, window=window, scale=float(np.float32(scale)))


def poison(seg, used):
    """NaN wherever no sequence has a row: other pages, and the rest of last pages."""
    page = seg["k"].shape[1]
    live = np.zeros(seg["k"].shape[:2], dtype=bool)
    for b, n in enumerate(used):
        for i in range(n):
            p = seg["table"][b, i // page]
            if 0 <= p < len(live):
                live[p, i % page] = True
    for name in ("k", "v"):
        scale = seg.get(name + "_scale")
        seg[name][~live] = 0x7F if scale is not None else np.nan
        if scale is not None:
            scale[~live] = np.nan


def rows_on(torch, ds4a, seg, pad_row=0, pad_page=0):
    """The segment on the device; rows and pages may be padded (NaN between)."""
    if seg is None:
        return None
    n, r, _ = seg["k"].shape

    def pool(a):
        big = torch.full((n, r * (D + pad_row) + pad_page), 0x7F if a.dtype == np.uint8 else float("nan"),
                         dtype=torch.uint8 if a.dtype == np.uint8 else torch.float16, device="cuda")
        view = big.as_strided((n, r, D), (big.shape[1], D + pad_row, 1))
        view.copy_(up(torch, a))
        return view
    k = pool(seg["k"])
    v = k if seg["v"] is seg["k"] else pool(seg["v"])
    ks, vs = up(torch, seg.get("k_scale")), up(torch, seg.get("v_scale"))
    return ds4a.PagedRows(k, v, up(torch, seg["table"]), k_scale=ks, v_scale=ks if v is k else vs)


def geometry(comp_rows, ratio, page, extra=3, window=128):
    """A token a few positions after its last compressed row, its raw rows kept by whole pages."""
    out = []
    for c in comp_rows:
        pos = c * ratio + min(extra, ratio - 1)
        first = max(0, pos + 1 - window) // page * page
        out.append((pos, pos + 1 - first, first, c))
    return out


def check_decode(got_o, got_lse, want, n_rows):
    o, lse, spread, reach = want
    e = 512 * 2.0 ** -23 * reach[:, None, None]
    bound = spread * (2.1 * F16 + np.expm1(2 * e)) + 2.0 ** -25
    got = got_o.astype(np.float64)
    assert np.isfinite(got).all()
    err = np.abs(got - o)
    assert (err <= bound).all(), f"worst {np.max(err / bound):.3f} of the bound, {err.max():.2e}"
    if got_lse is not None:
        fin = np.isfinite(lse)
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
        lb = e[:, :, 0] + (np.asarray(n_rows)[:, None] / 128 + 40) * 2.0 ** -23 + np.abs(np.where(fin, lse, 0)) * 2.0 ** -22
        el = np.abs(np.where(fin, got_lse.astype(np.float64) - np.where(fin, lse, 0), 0))
        assert (el <= lb).all(), f"lse worst {np.max(el / lb):.3f} of the bound"


def case(rng, comp_rows, ratio, page, fp8_rows, shared, window=128, absent=()):
    geom = geometry(comp_rows, ratio, page, window=window)
    n = len(comp_rows)
    comp = make(rng, n, comp_rows, page, fp8_rows, shared, absent)
    raw = make(rng, n, [g[1] for g in geom], page, fp8_rows, shared)
    poison(comp, comp_rows)
    poison(raw, [g[1] for g in geom])
    q = rng.standard_normal((n, H, D)).astype(np.float16)
    return geom, q, raw, comp


DECODE = [  # compressed rows per sequence, ratio, page rows, fp8, K = V, window
    ([0], 4, 16, False, False, 128),
    ([1], 1, 1, False, False, 128),
    ([256], 128, 64, False, False, 128),
    ([0, 5, 127, 128, 129, 1000], 4, 16, False, True, 128),
    ([3, 700, 0, 64], 4, 100, False, False, 1),
    ([500, 20, 333], 4, 7, False, True, 300),
    ([4000], 4, 128, False, False, 128),
    ([256], 128, 64, True, False, 128),
    ([0, 5, 127, 128, 129, 1000], 4, 16, True, True, 128),
    ([3, 700, 0, 64], 4, 100, True, False, 200),
    ([4100, 40], 4, 256, True, True, 128),
]


@pytest.mark.parametrize("k", range(len(DECODE)))
def test_decode_matches_the_oracle(torch, ds4a, k):
    comp_rows, ratio, page, f8, shared, window = DECODE[k]
    rng = np.random.default_rng(100 + k)
    geom, q, raw, comp = case(rng, comp_rows, ratio, page, f8, shared, window)
    shape = shape_of(ratio, window)
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    n_rows = [window + c for c in comp_rows]
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), n_rows)


@pytest.mark.parametrize("f8", [False, True])
def test_decode_many_ragged_sequences(torch, ds4a, f8):
    """More tiles than CTAs, sequences cut at CTA borders, sequences without rows."""
    rng = np.random.default_rng(7)
    comp_rows = [int(x) for x in rng.integers(0, 900, 70)]
    geom, q, raw, comp = case(rng, comp_rows, 4, 32, f8, True)
    for b in (0, 13, 69):  # nothing visible: no rows at all
        geom[b] = (geom[b][0], 0, 0, 0)
    shape = shape_of()
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    want = paged.decode(shape, geom, q, raw, comp)
    check_decode(host(o), host(lse), want, [c + 128 for c in comp_rows])
    for b in (0, 13, 69):
        assert (host(o)[b] == 0).all() and np.isneginf(host(lse)[b]).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [16, 64, 128, 24])
def test_decode_long_ragged_batches_back_to_back(torch, ds4a, page, f8):
    """Several tiles per CTA, whole tiles and gathered ones in turn, calls queued without a wait: the same bits
    each time, and the oracle's values."""
    rng = np.random.default_rng(16)
    comp_rows = [int(x) for x in rng.integers(300, 2000, 60)]
    geom, q, raw, comp = case(rng, comp_rows, 4, page, f8, True)
    shape, g, qd = shape_of(), up(torch, np.array(geom, dtype=np.int32)), up(torch, q)
    r, c = rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp)
    ws = torch.empty(ds4a.decode_paged_workspace_bytes(60), dtype=torch.uint8, device="cuda")
    outs = [ds4a.attn_decode_paged(shape, g, qd, r, c, want_lse=True, workspace=ws) for _ in range(30)]
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    few = [0, 7, 31, 59]
    want = [paged.decode(shape, [geom[b]], q[b:b + 1], dict(raw, table=raw["table"][b:b + 1]),
                         dict(comp, table=comp["table"][b:b + 1])) for b in few]
    for b, w in zip(few, want):
        check_decode(host(outs[0][0])[b:b + 1], host(outs[0][1])[b:b + 1], w, [comp_rows[b] + 128])


def test_decode_more_sequences_than_threads(torch, ds4a):
    """1300 sequences of a few rows: the plan runs over several rounds of the block."""
    rng = np.random.default_rng(8)
    comp_rows = [int(x) for x in rng.integers(0, 4, 1300)]
    geom, q, raw, comp = case(rng, comp_rows, 128, 4, False, True, window=2)
    shape = shape_of(128, 2)
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [4] * 1300)


@pytest.mark.parametrize("f8", [False, True])
def test_decode_absent_pages(torch, ds4a, f8):
    """Pages named by nothing: -1, n_pages and far beyond; a whole sequence of them; whole tiles of them."""
    rng = np.random.default_rng(9)
    geom, q, raw, comp = case(rng, [300, 260, 200], 4, 16, f8, False)
    n_pages = len(comp["k"])
    comp["table"][0, [0, 5, 18]] = [-1, n_pages, 2 ** 31 - 1]
    comp["table"][1, :] = -7
    comp["table"][2, :8] = -2 ** 31  # the first 128 compressed rows
    raw["table"][1, :] = n_pages + 100000
    shape = shape_of()
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    want = paged.decode(shape, geom, q, raw, comp)
    assert np.isneginf(want[1][1]).all()
    check_decode(host(o), host(lse), want, [428] * 3)


@pytest.mark.parametrize("f8", [False, True])
def test_decode_strides_and_untouched_rows(torch, ds4a, f8):
    """Padded rows, pages, tables, tokens; more outputs and tables than sequences: the rest stays as it was."""
    rng = np.random.default_rng(10)
    comp_rows = [200, 31]
    geom, q, raw, comp = case(rng, comp_rows, 4, 12, f8, False)
    shape = shape_of()
    qq = torch.full((4, H + 3, D), float("nan"), dtype=torch.float16, device="cuda")
    qq[:2, :H] = up(torch, q)
    out = torch.full((5, H + 1, D), 7.0, dtype=torch.float16, device="cuda")
    segs = []
    for s in (raw, comp):
        r = rows_on(torch, ds4a, s, pad_row=16, pad_page=48)
        wide = torch.full((4, s["table"].shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
        wide[:2, :s["table"].shape[1]] = up(torch, s["table"])
        segs.append(ds4a.PagedRows(r.k, r.v, wide[:, :s["table"].shape[1]], k_scale=r.k_scale, v_scale=r.v_scale))
    ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), qq[:2, :H], *segs, out=out[:2, :H])
    check_decode(host(out[:2, :H]), None, paged.decode(shape, geom, q, raw, comp), [c + 128 for c in comp_rows])
    assert (out[2:] == 7).all() and (out[:, H:] == 7).all()


def test_decode_one_segment_only(torch, ds4a):
    rng = np.random.default_rng(11)
    geom, q, raw, comp = case(rng, [150, 3], 4, 16, False, True)
    shape, g = shape_of(), up(torch, np.array(geom, dtype=np.int32))
    for r, c in ((raw, None), (None, comp)):
        o, lse = ds4a.attn_decode_paged(shape, g, up(torch, q), rows_on(torch, ds4a, r), rows_on(torch, ds4a, c),
                                        want_lse=True)
        check_decode(host(o), host(lse), paged.decode(shape, geom, q, r, c), [278, 131])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("n", [2, 31, 32, 33, 64, 65, 100, 153, 512, 513])
def test_decode_batches_of_every_plan(torch, ds4a, n, f8):
    """Batches on both sides of each way of sharing out the tiles, with empty sequences first, between and last."""
    rng = np.random.default_rng(60 + n)
    comp_rows = [int(x) for x in rng.integers(0, 500 if n < 60 else 150, n)]
    geom, q, raw, comp = case(rng, comp_rows, 4, 8, f8, True, window=16)
    for b in {0, n // 2, n - 1} if n > 2 else {1}:
        geom[b] = (geom[b][0], 0, 0, 0)
    shape = shape_of(4, 16)
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [c + 16 for c in comp_rows])


@pytest.mark.parametrize("short,long", [(149, 48), (150, 32), (60, 200), (0, 40), (7, 300), (31, 90), (400, 64)])
def test_decode_shares_one_long_sequence_out(torch, ds4a, short, long):
    """Many sequences of one tile and a long one: no CTA has more tiles of it than the average and two, or than
    three where that is two.  (What a call leaves behind the partial results in its workspace: per sequence the first
    slot and the number of slots.)"""
    rng = np.random.default_rng(65)
    n = short + 1
    comp_rows = [128] * short + [128 * long]
    comp_rows[short // 2], comp_rows[-1] = comp_rows[-1], comp_rows[short // 2]
    pages = 16  # of 64 rows, shared by all tables
    k = rng.standard_normal((pages, 64, D)).astype(np.float16)
    table = rng.integers(0, pages, (n, 2 * long)).astype(np.int32)
    geom = [(4 * c, 0, 0, c) for c in comp_rows]
    q = rng.standard_normal((n, H, D)).astype(np.float16)
    shape = shape_of()
    ws = torch.zeros(ds4a.decode_paged_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q), None,
                                    ds4a.PagedRows(up(torch, k), None, up(torch, table)), want_lse=True, workspace=ws)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    average = -(-(short + long) // ctas)
    plan = host(ws[(n + ctas) * H * (4 * D + 8):][:8 * n].view(torch.int32)).reshape(n, 2)
    assert -(-long // plan[short // 2, 1]) <= average + min(2, average - 1), plan[short // 2]
    seg = dict(k=k, v=k, table=table)
    few = sorted({0, short // 2, n - 1})
    want = paged.decode(shape, [geom[b] for b in few], q[few], None, dict(seg, table=table[few]))
    check_decode(host(o)[few], host(lse)[few], want, [comp_rows[b] for b in few])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("pad_row", [D, 4 * D])
def test_decode_rows_of_interleaved_layers(torch, ds4a, pad_row, f8):
    """Rows far apart (a pool that holds several layers' rows side by side), NaN between them."""
    rng = np.random.default_rng(61)
    comp_rows = [1500, 700, 140]
    geom, q, raw, comp = case(rng, comp_rows, 4, 64, f8, True)
    shape = shape_of()
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw, pad_row=pad_row),
                                    rows_on(torch, ds4a, comp, pad_row=pad_row), want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [c + 128 for c in comp_rows])


@pytest.mark.parametrize("scale", [1e25, 1e33])
def test_decode_of_one_row_is_its_value(torch, ds4a, scale):
    """However low the row's score: a softmax over one row is 1."""
    rng = np.random.default_rng(62)
    seg = make(rng, 1, [1], 16)
    q = torch.from_numpy(-np.repeat(seg["k"][seg["table"][0, 0], 0][None, None], H, 1)).cuda()
    geom = torch.tensor([[7, 0, 0, 1]], dtype=torch.int32, device="cuda")
    o, lse = ds4a.attn_decode_paged(shape_of(scale=scale), geom, q, None, rows_on(torch, ds4a, seg), want_lse=True)
    want = seg["v"][seg["table"][0, 0], 0]
    assert np.array_equal(host(o)[0], np.repeat(want[None], H, 0))
    k = seg["k"][seg["table"][0, 0], 0].astype(np.float64)
    assert np.abs(host(lse)[0] / (-float(np.float32(scale)) * (k * k).sum()) - 1).max() <= 516 * 2.0 ** -23  # products and sums, and eight roundings


@pytest.mark.parametrize("rows", [[100], [4000], [100] * 200, [700] * 60, [2000] * 60, [5000] * 9])
@pytest.mark.parametrize("f8", [False, True])
def test_decode_hides_no_nan(torch, ds4a, rows, f8):
    """A NaN in a head's query makes that head's output and log-sum-exp NaN, one in a row that is seen every head's,
    whether one CTA has the whole sequence or several share it; other heads and sequences stay as they are."""
    rng = np.random.default_rng(66)
    n, page = len(rows), 64
    pages = -(-max(rows) // page)
    k = up(torch, rng.integers(0, 120, (pages + 1, page, D)).astype(np.uint8) if f8 else
           rng.standard_normal((pages + 1, page, D)).astype(np.float16))
    ks = torch.full((pages + 1, page), 0.01, device="cuda") if f8 else None
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n, 1)
    b, row = n // 2, rows[n // 2] - 30
    k[-1] = k[row // page]
    if ks is not None:
        ks[-1] = ks[row // page]
    table[b, row // page] = pages  # sequence b's alone
    seg = ds4a.PagedRows(k, None, table, k_scale=ks)
    geom = up(torch, np.array([(4 * r, 0, 0, r) for r in rows], dtype=np.int32))
    q = up(torch, rng.standard_normal((n, H, D)).astype(np.float16))
    o, lse = ds4a.attn_decode_paged(shape_of(), geom, q, None, seg, want_lse=True)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    bad = q.clone()
    bad[b, 5, 17] = float("nan")
    o2, lse2 = ds4a.attn_decode_paged(shape_of(), geom, bad, None, seg, want_lse=True)
    assert torch.isnan(o2[b, 5]).all() and torch.isnan(lse2[b, 5])
    o2[b, 5], lse2[b, 5] = o[b, 5], lse[b, 5]
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    k[-1, row % page, 9] = 0x7F if f8 else float("nan")
    o3, lse3 = ds4a.attn_decode_paged(shape_of(), geom, q, None, seg, want_lse=True)
    assert torch.isnan(o3[b]).all() and torch.isnan(lse3[b]).all()
    o3[b], lse3[b] = o[b], lse[b]
    assert torch.equal(o3, o) and torch.equal(lse3, lse)


@pytest.mark.parametrize("n", [1, 40, 70])
def test_decode_without_any_segment(torch, ds4a, n):
    q = torch.ones((n, H, D), dtype=torch.float16, device="cuda")
    geom = torch.full((n, 4), 9, dtype=torch.int32, device="cuda")
    o, lse = ds4a.attn_decode_paged(shape_of(), geom, q, None, None, out=torch.full_like(q, 3.0), want_lse=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_decode_pages_past_32_bit_offsets(torch, ds4a):
    """A 5 GB pool whose used pages lie at its end, read through both tables by two sequences (shared pages)."""
    rng = np.random.default_rng(12)
    page, n_pages = 64, 80000
    rows = rng.standard_normal((6, page, D)).astype(np.float16)
    k = torch.empty((n_pages, page, D), dtype=torch.float16, device="cuda")
    k[-6:] = up(torch, rows)
    table = np.array([[n_pages - 1, n_pages - 3, n_pages - 2, n_pages - 6], [n_pages - 3, n_pages - 3, -1, -1]],
                     dtype=np.int32)
    geom = [(4000, 0, 0, 250), (4000, 0, 0, 100)]
    small = dict(k=rows, v=rows, table=np.where(table >= 0, table - (n_pages - 6), -1))
    q = rng.standard_normal((2, H, D)).astype(np.float16)
    shape = shape_of()
    seg = ds4a.PagedRows(k, None, up(torch, table))
    g = up(torch, np.array(geom, dtype=np.int32))
    o, lse = ds4a.attn_decode_paged(shape, g, up(torch, q), None, seg, want_lse=True)
    want = paged.decode(shape, geom, q, None, small)
    check_decode(host(o), host(lse), want, [250, 100])
    w = ds4a.attn_weights_paged(shape, g, up(torch, q), seg, lse)
    np.testing.assert_allclose(host(w).sum(1), 64.0, rtol=1e-3)
    slots = torch.tensor([(n_pages - 1) * page + 5], dtype=torch.int32, device="cuda")
    new = up(torch, rng.standard_normal((1, D)).astype(np.float16))
    ds4a.append_paged(seg, new, None, slots)
    assert torch.equal(k[-1, 5], new[0])
    del k, seg


@pytest.mark.parametrize("exponent", [-30, -12, 0, 9])
def test_decode_e4m3_scales_of_any_size(torch, ds4a, exponent):
    """V scales from 2^-30 to 2^9 of the usual: the output keeps its relative
    precision; rows of scale 0 keep their weight and have no value."""
    rng = np.random.default_rng(13)
    geom, q, raw, comp = case(rng, [600], 4, 16, True, False)
    for s in (raw, comp):
        s["v_scale"][:] = s["v_scale"] * np.float32(2.0 ** exponent) * np.exp2(rng.integers(-3, 4, s["v_scale"].shape))
    comp["v_scale"][:, 3] = 0.0
    shape = shape_of()
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [728])


def test_decode_large_scores_move_the_reference(torch, ds4a):
    """Scores that grow along the rows by far more than 2^8, and rows of opposite sign."""
    rng = np.random.default_rng(14)
    geom, q, raw, comp = case(rng, [1500], 4, 64, False, True)
    grow = np.linspace(0.1, 6.0, comp["k"].shape[0] * 64).astype(np.float16).reshape(-1, 64, 1)
    comp["k"][:] = comp["k"] * grow
    comp["v"] = comp["k"]
    shape = shape_of()
    o, lse = ds4a.attn_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                    rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [1628])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("n_seq", [1, 64])
@pytest.mark.parametrize("below", [12.3, 20.7, 24.6, 25.0, 25.5, 28.3])
def test_decode_of_a_long_tail_under_one_row(torch, ds4a, below, n_seq, f8):
    """One row on top whose value is 0, and 65,535 rows of value 1, each with 2^-below of its weight: the output is
    the tail's share.  Scores are single products (exact but for the rounding of the scale and of the product, 2^-23
    of a score: 2^-18 of a weight).  A weight's rounding is at most 2^-11 of it, or half a step of fp16's smallest
    numbers, where the largest weight counts as 2^10: 2^-35 of that one; the output is rounded (2^-11, or 2^-25)."""
    n, page = 65536, 128
    k = torch.zeros((n // page, page, D), dtype=torch.uint8 if f8 else torch.float16, device="cuda")
    v = torch.full_like(k, 0x38 if f8 else 1.0)  # 0x38: the E4M3 code of 1
    k[0, 5, 7] = 0x50 if f8 else 8.0             # 8
    v[0, 5] = 0
    one = torch.ones((n // page, page), device="cuda") if f8 else None
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    q = torch.zeros((n_seq, H, D), dtype=torch.float16, device="cuda")
    q[:, :, 7] = 1
    geom = torch.tensor([[4 * n, 0, 0, n]] * n_seq, dtype=torch.int32, device="cuda")
    shape = shape_of(scale=below * np.log(2.0) / 8)
    o, lse = ds4a.attn_decode_paged(shape, geom, q, None, ds4a.PagedRows(k, v, table, k_scale=one, v_scale=one),
                                    want_lse=True)
    e = np.exp(-8 * np.float64(shape["scale"]))
    want = (n - 1) * e / (1 + (n - 1) * e)
    bound = want * (2.0 ** -11 + max(2.0 ** -11, 2.0 ** -35 / e) + 2.0 ** -17) + 2.0 ** -25
    got = host(o).astype(np.float64)
    assert np.abs(got - want).max() <= bound, f"{got.min()} .. {got.max()}, {want} +- {bound}"
    assert np.abs(host(lse) - (8 * np.float64(shape["scale"]) + np.log1p((n - 1) * e))).max() <= \
        (n / 128 + 40) * 2.0 ** -23 + 32 * 2.0 ** -22


@pytest.mark.parametrize("base", range(4))
def test_decode_scores_a_step_apart_stay_finite(torch, ds4a, base):
    """Scores near 2^27, where fp32 numbers are 16 apart: a row one step above a tile's largest, in a later tile,
    is the new reference, not a weight of 2^16.  (Whichever scores round alike, the output lies between the values.)"""
    k = torch.zeros((2, 128, D), dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    k[:, :, 0], k[:, :, 1] = 6144.0, float(base)  # 2048 * 6144 + base
    k[1, 9, 1] = base + 1.0
    v[1, 9] = 2.0
    q = torch.zeros((8, H, D), dtype=torch.float16, device="cuda")
    q[:, :, 0], q[:, :, 1] = 2048.0, 1.0
    table = torch.arange(2, dtype=torch.int32, device="cuda").repeat(8, 1)
    geom = torch.tensor([[1024, 0, 0, 256]] * 8, dtype=torch.int32, device="cuda")
    o, lse = ds4a.attn_decode_paged(shape_of(scale=16 * np.log(2.0)), geom, q, None, ds4a.PagedRows(k, v, table),
                                    want_lse=True)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert (o >= 1).all() and (o <= 2).all()


def test_decode_equals_batched_decode_and_itself(torch, ds4a):
    """The batched decode over the same rows, gathered; the same call twice, bit for bit, on a dirty workspace."""
    rng = np.random.default_rng(15)
    comp_rows = [512, 300, 40]
    geom, q, raw, comp = case(rng, comp_rows, 4, 16, False, False)
    shape, g = shape_of(), up(torch, np.array(geom, dtype=np.int32))
    args = (shape, g, up(torch, q), rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp))
    ws = torch.full((ds4a.decode_paged_workspace_bytes(3),), 0xFF, dtype=torch.uint8, device="cuda")
    o1, l1 = ds4a.attn_decode_paged(*args, want_lse=True, workspace=ws)
    o1, l1 = o1.clone(), l1.clone()
    o2, l2 = ds4a.attn_decode_paged(*args, want_lse=True, workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    dense = []
    for s, n in ((raw, max(x[1] for x in geom)), (comp, 512)):
        for w in ("k", "v"):
            dense.append(up(torch, np.stack([paged.segment_rows(s, b, n, w)[0] for b in range(3)]).astype(np.float16)))
    # rows outside a sequence's own must be finite there
    ob, lb = ds4a.attn_decode_batch(shape, g, up(torch, q), *[torch.nan_to_num(d) for d in dense], want_lse=True)
    assert (o1.float() - ob.float()).abs().max() <= 2e-3 and (l1 - lb).abs().max() <= 1e-3


# ------------------------------------------------------------------ received weights

@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("rows,page", [([1], 1), ([0, 128, 129, 700], 16), ([2049], 100), (list(range(40)) * 5, 8)])
def test_weights_match_the_oracle(torch, ds4a, f8, rows, page):
    rng = np.random.default_rng(20 + page)
    n = len(rows)
    geom = geometry(rows, 4, page)
    comp = make(rng, n, rows, page, f8, True, absent=((n - 1, 0),) if n > 3 else ())
    poison(comp, rows)
    q = rng.standard_normal((n, H, D)).astype(np.float16)
    shape = shape_of()
    _, lse, _, reach = paged.decode(shape, geom, q, None, comp)
    lse = (lse + 0.3).astype(np.float32)
    lse[:, 5] = -np.inf
    cap = paged.capacity(comp)
    before = rng.random((n, cap)).astype(np.float32)
    out = torch.full((n + 1, cap + 4), 5.0, device="cuda")
    ds4a.attn_weights_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q), rows_on(torch, ds4a, comp),
                            up(torch, lse), weights=up(torch, before), decay=0.9, out=out[:n, :cap])
    want = paged.weights(shape, geom, q, comp, lse, before, 0.9)
    got = host(out)
    assert (got[n:] == 5).all() and (got[:, cap:] == 5).all()
    written = ~np.isnan(want)
    assert (got[:n, :cap][~written] == 5).all()
    size = 4 * (reach + np.abs(np.where(np.isfinite(lse), lse, 0)).max(1) + 1)
    rel = np.expm1(512 * 2.0 ** -23 * reach) + (64 + size) * 2.0 ** -23
    w0, b0 = np.where(written, want, 0), before
    assert (np.abs(got[:n, :cap] - w0)[written] <= (rel[:, None] * w0 + 2.0 ** -22 * b0)[written]).all()


def test_weights_in_place_and_without_history(torch, ds4a):
    rng = np.random.default_rng(30)
    geom = geometry([300, 77], 4, 16)
    comp = make(rng, 2, [300, 77], 16)
    q = rng.standard_normal((2, H, D)).astype(np.float16)
    shape, g, qd, seg = shape_of(), up(torch, np.array(geom, dtype=np.int32)), up(torch, q), rows_on(torch, ds4a, comp)
    _, lse = ds4a.attn_decode_paged(shape, g, qd, None, seg, want_lse=True)
    w = ds4a.attn_weights_paged(shape, g, qd, seg, lse)
    np.testing.assert_allclose(host(w).sum(1), 64.0, rtol=2e-4)
    once = w.clone()
    ds4a.attn_weights_paged(shape, g, qd, seg, lse, weights=w, decay=0.5, out=w)
    np.testing.assert_allclose(host(w), 1.5 * host(once), rtol=1e-6)


# ------------------------------------------------------------------ eviction

def run_evict(torch, ds4a, rng, rows, page, keep, f8=False, shared=False, ids=None, first=0, recent=0, w=None,
              in_place=False, absent=(), ratio=4):
    n = len(rows)
    geom = [(r * ratio, 0, 0, r) for r in rows]
    seg = make(rng, n, rows, page, f8, shared, absent)
    cap = paged.capacity(seg)
    if w is None:
        w = rng.integers(0, 50, (n, cap)).astype(np.float32)
    dev = rows_on(torch, ds4a, seg)
    g = up(torch, np.array(geom, dtype=np.int32))
    wd, idd = up(torch, w), up(torch, ids)
    w_out = wd if in_place else torch.full((n, cap), -1.0, device="cuda")
    i_out = None if ids is None else (idd if in_place else torch.full((n, cap), -1, dtype=torch.int32, device="cuda"))
    ws = torch.full((ds4a.evict_paged_workspace_bytes(n, keep),), 0xEE, dtype=torch.uint8, device="cuda")
    kept, n_out = ds4a.evict_paged(shape_of(ratio), g, dev, wd, keep, n_first=first, n_recent=recent, ids=idd,
                                   weights_out=w_out, ids_out=i_out, n_out=g[:, 3] if in_place else None, workspace=ws)
    want = paged.evict(dict(ratio=ratio), geom, w, ids, keep, first, recent, cap)
    kept, n_out = host(kept), host(n_out)
    if in_place:
        assert np.array_equal(host(g)[:, 3], n_out) and np.array_equal(host(g)[:, :3], np.array(geom)[:, :3])
    for b, (no, kp) in enumerate(want):
        assert n_out[b] == no and np.array_equal(kept[b, :no], kp) and (kept[b, no:] == -1).all(), b
        np.testing.assert_array_equal(host(w_out)[b, :no], w[b][kp])
        rest = w[b, no:] if in_place else np.full(cap - no, -1)
        np.testing.assert_array_equal(host(w_out)[b, no:], rest)
        if ids is not None:
            np.testing.assert_array_equal(host(i_out)[b, :no], ids[b][kp])
        paged.move_rows(seg, b, kp)
    assert np.array_equal(host(dev.k).view(np.uint8), seg["k"].view(np.uint8))
    assert np.array_equal(host(dev.v).view(np.uint8), seg["v"].view(np.uint8))
    if f8:
        assert np.array_equal(host(dev.k_scale), seg["k_scale"]) and np.array_equal(host(dev.v_scale), seg["v_scale"])


@pytest.mark.parametrize("rows,page,keep", [
    ([1], 1, 1), ([2], 1, 1), ([5, 0, 1, 9], 4, 3), ([100, 1000, 33], 16, 33), ([700], 100, 699), ([700], 100, 1),
    ([1025] * 5, 64, 1024), ([3000, 2999], 7, 1500), ([64, 64], 64, 64), ([40], 16, 1000)])
@pytest.mark.parametrize("f8,shared", [(False, False), (True, True), (True, False)])
def test_evict_matches_the_oracle(torch, ds4a, rows, page, keep, f8, shared):
    run_evict(torch, ds4a, np.random.default_rng(sum(rows) + page), rows, page, keep, f8, shared)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_protects_by_id(torch, ds4a, in_place):
    rng = np.random.default_rng(41)
    rows = [500, 300]
    ids = np.stack([rng.permutation(512) for _ in rows]).astype(np.int32)
    run_evict(torch, ds4a, rng, rows, 32, 200, ids=ids, first=4, recent=64, in_place=in_place)
    run_evict(torch, ds4a, rng, rows, 32, 50, ids=ids, first=4, recent=64, in_place=in_place)  # more protected than kept
    run_evict(torch, ds4a, rng, rows, 32, 450, first=2, recent=10 ** 6, in_place=in_place)


def test_evict_at_the_ends_of_the_integers(torch, ds4a):
    """The last position an int32 holds, ids at both ends, and the largest n_recent."""
    w = np.arange(64, dtype=np.float32)[None]
    ids = np.linspace(-2 ** 31, 2 ** 31 - 1, 64).astype(np.int64).astype(np.int32)[None]
    seg = make(np.random.default_rng(0), 1, [64], 16)
    for pos, recent, first in ((2 ** 31 - 1, 0, 0), (2 ** 31 - 1, 2 ** 31 - 1, 0), (0, 2 ** 31 - 1, 2 ** 31 - 1), (5, 3, 0)):
        geom = [(pos, 0, 0, 64)]
        kept, n_out = ds4a.evict_paged(shape_of(1), up(torch, np.array(geom, dtype=np.int32)), rows_on(torch, ds4a, seg),
                                       up(torch, w), 20, n_first=first, n_recent=recent, ids=up(torch, ids))
        (no, kp), = paged.evict(dict(ratio=1), geom, w, ids, 20, first, recent, 64)
        assert host(n_out)[0] == no and np.array_equal(host(kept)[0], kp), (pos, recent)


@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "inf", "subnormal", "negative"])
def test_evict_weights_of_every_kind(torch, ds4a, kind):
    rng = np.random.default_rng(42)
    w = rng.standard_normal((2, 1008)).astype(np.float32)
    if kind == "equal":
        w[:] = 1.25
    elif kind == "zeros":
        w = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0).astype(np.float32)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.7] = np.nan
        w[rng.random(w.shape) < 0.1] = -np.inf
    elif kind == "inf":
        w[rng.random(w.shape) < 0.5] = np.inf
    elif kind == "subnormal":
        w = (rng.integers(-40, 40, w.shape) * 2.0 ** -149).astype(np.float32)
    else:
        w = -np.abs(w)
    run_evict(torch, ds4a, rng, [1000, 777], 16, 500, w=w)


@pytest.mark.parametrize("rows,keep", [([20000, 9000], 7000), ([40000], 39000), ([70001], 11)])
def test_evict_long_sequences(torch, ds4a, rows, keep):
    """Clusters of CTAs share a sequence; E4M3 rows to keep the pool small."""
    rng = np.random.default_rng(43)
    page = 128
    geom = [(4 * r, 0, 0, r) for r in rows]
    per = [-(-r // page) for r in rows]
    table = np.full((len(rows), max(per)), -1, dtype=np.int32)
    order, at = rng.permutation(sum(per)), 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    k = torch.randint(0, 120, (sum(per), page, D), dtype=torch.uint8, device="cuda")
    ks = torch.rand((sum(per), page), device="cuda")
    k0, ks0 = k.clone(), ks.clone()
    cap = max(per) * page
    w = rng.integers(0, 300, (len(rows), cap)).astype(np.float32)
    seg = ds4a.PagedRows(k, None, up(torch, table), k_scale=ks)
    wd = up(torch, w)
    kept, n_out = ds4a.evict_paged(shape_of(), up(torch, np.array(geom, dtype=np.int32)), seg, wd, keep, n_recent=50)
    want = paged.evict(dict(ratio=4), geom, w, None, keep, 0, 50, cap)
    for b, (no, kp) in enumerate(want):
        assert host(n_out)[b] == no and np.array_equal(host(kept)[b, :no], kp)
        np.testing.assert_array_equal(host(wd)[b, :no], w[b][kp])
        src = torch.from_numpy(kp.copy()).cuda()
        dst = torch.arange(no, device="cuda")
        t = seg.table[b].long()
        assert torch.equal(k[t[dst // page], dst % page], k0[t[src // page], src % page])
        assert torch.equal(ks[t[dst // page], dst % page], ks0[t[src // page], src % page])


def test_evict_the_longest_lists(torch, ds4a):
    """More keys than a cluster's shared memory holds: ranks are taken from the weights each time."""
    n, page = 850000, 512
    pages = -(-n // page)
    k = torch.zeros((pages, page, D), dtype=torch.uint8, device="cuda")
    ks = torch.arange(pages * page, dtype=torch.float32, device="cuda").view(pages, page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    g = torch.tensor([[4 * n, 0, 0, n]], dtype=torch.int32, device="cuda")
    w = torch.randint(0, 1000, (1, pages * page), device="cuda").float()
    keep = 500000
    want = torch.sort(w[0, :n], descending=True, stable=True).indices[:keep].sort().values
    w0 = w.clone()
    kept, n_out = ds4a.evict_paged(shape_of(), g, ds4a.PagedRows(k, None, table, k_scale=ks), w, keep)
    assert n_out.item() == keep
    assert torch.equal(kept[0].long().sort().values, want)
    stay = want[want < keep]
    assert torch.equal(kept[0, stay].long(), stay)
    assert torch.equal(w[0, :keep], w0[0, kept[0].long()])
    assert torch.equal(ks.view(-1)[:keep], kept[0].float())


def test_evict_absent_pages_move_nothing(torch, ds4a):
    rng = np.random.default_rng(44)
    run_evict(torch, ds4a, rng, [100, 90], 10, 40, absent=((0, 1), (0, 7), (1, 8)))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("n,page,pages", [(1, 1, 1), (5, 7, 3), (64, 16, 40), (700, 100, 9)])
def test_append_matches_the_oracle(torch, ds4a, f8, shared, n, page, pages):
    rng = np.random.default_rng(50 + n)
    seg = make(rng, 1, [page * pages], page, f8, shared)
    dev = rows_on(torch, ds4a, seg, pad_row=16, pad_page=32)
    new = (rng.standard_normal((n, 2, D)) * np.exp(rng.standard_normal((n, 1, 1)))).astype(np.float16)
    new[0] = 0
    new[-1, :, ::3] = 65504
    slots = rng.permutation(page * pages)[:n].astype(np.int64)
    slots[::5] = rng.choice([-1, page * pages, 2 ** 31 - 1, -2 ** 31], len(slots[::5]))
    buf = up(torch, new)
    ds4a.append_paged(dev, buf[:, 0], buf[:, 1], up(torch, slots.astype(np.int32)))
    for i, s in enumerate(slots):
        if 0 <= s < page * pages:
            for j, name in enumerate(("k",) if shared else ("k", "v")):
                row = new[i:i + 1, j]
                if f8:
                    c, sc = fp8.quantize_rows(row)
                    seg[name][s // page, s % page], seg[name + "_scale"][s // page, s % page] = c[0], sc[0]
                else:
                    seg[name][s // page, s % page] = row[0]
    for name in ("k", "v"):
        assert np.array_equal(host(getattr(dev, name)).view(np.uint8), seg[name].view(np.uint8))
        if f8:
            assert np.array_equal(host(getattr(dev, name + "_scale")), seg[name + "_scale"])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("page,pages,slots", [(1, 1, [0]), (4, 2, [7]), (5, 3, [14, -1, 0, 6, 15, 5])])
def test_append_writes_one_row_and_rows_of_zeros(torch, ds4a, f8, shared, page, pages, slots):
    """A single row, the pool's first and last slots, and (first) a row of zeros: scale 0, codes 0 over what the slot
    held; the other slots keep their bytes."""
    rng = np.random.default_rng(58)
    seg = make(rng, 1, [page * pages], page, f8, shared)
    for zero in (False, True):
        dev = rows_on(torch, ds4a, seg)
        new = rng.standard_normal((len(slots), 2, D)).astype(np.float16)
        if zero:
            new[0] = 0
        buf = up(torch, new)
        before = host(dev.k).copy()
        ds4a.append_paged(dev, buf[:, 0], buf[:, 1], up(torch, np.array(slots, dtype=np.int32)))
        kept = [s for s in slots if 0 <= s < page * pages]
        for i, s in enumerate(slots):
            if s not in kept:
                continue
            for j, name in enumerate(("k",) if shared else ("k", "v")):
                at, row = (s // page, s % page), new[i:i + 1, j]
                if f8:
                    c, sc = fp8.quantize_rows(row)
                    seg[name][at], seg[name + "_scale"][at] = c[0], sc[0]
                    assert not (zero and i == 0) or (sc[0] == 0 and (c == 0).all())
                else:
                    seg[name][at] = row[0]
        assert len(kept) >= 1 and not np.array_equal(host(dev.k).view(np.uint8), before.view(np.uint8))
        for name in ("k", "v"):
            assert np.array_equal(host(getattr(dev, name)).view(np.uint8), seg[name].view(np.uint8))
            if f8:
                assert np.array_equal(host(getattr(dev, name + "_scale")), seg[name + "_scale"])


def test_append_to_one_row_pool_with_two_scale_arrays(torch, ds4a):
    """K = V rows with a scale array each: both get the new row's scale, and a decode that reads them sees it."""
    rng = np.random.default_rng(57)
    page, pages = 4, 3
    seg = make(rng, 1, [page * pages], page, True, True)
    seg["v_scale"] = seg["k_scale"] * np.float32(3)
    k = up(torch, seg["k"])
    dev = ds4a.PagedRows(k, k, up(torch, seg["table"]), k_scale=up(torch, seg["k_scale"]),
                         v_scale=up(torch, seg["v_scale"]))
    new = (5 * rng.standard_normal((5, D))).astype(np.float16)
    new[2] = 0
    slots = np.array([0, 7, 11, -1, 4])
    ds4a.append_paged(dev, up(torch, new), None, up(torch, slots.astype(np.int32)))
    codes, scale = fp8.quantize_rows(new)
    for i, s in enumerate(slots):
        if s >= 0:
            at = (s // page, s % page)
            seg["k"][at], seg["k_scale"][at], seg["v_scale"][at] = codes[i], scale[i], scale[i]
    for name in ("k", "k_scale", "v_scale"):
        assert np.array_equal(host(getattr(dev, name)), seg[name]), name
    geom, q = [(4 * 12, 0, 0, 12)], rng.standard_normal((1, H, D)).astype(np.float16)
    seg["v"] = seg["k"]
    o, lse = ds4a.attn_decode_paged(shape_of(), up(torch, np.array(geom, dtype=np.int32)), up(torch, q), None, dev,
                                    want_lse=True)
    check_decode(host(o), host(lse), paged.decode(shape_of(), geom, q, None, seg), [12])


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,width,group", [
    (1, 8, 0), (3, 8, 32), (5, 136, 64), (9, 512, 0), (2, 512, 128), (7, 520, 0), (4, 1000, 256), (1, 4096, 128),
    (3, 7168, 0), (2, 8192, 32), (2, 8200, 0), (2, 16384, 128), (1, 20000, 64), (1, 32768, 0)])
def test_norm_matches_the_oracle(torch, ds4a, f32, residual, n, width, group):
    rng = np.random.default_rng(60 + width)
    dt = np.float32 if f32 else np.float16
    x = (rng.standard_normal((n, width)) * np.exp2(rng.integers(-6, 7, (n, 1)))).astype(dt)
    r = rng.standard_normal((n, width)).astype(dt) if residual else None
    w = (1 + 0.3 * rng.standard_normal(width)).astype(np.float32)
    w[:: 5] = 0
    if group and width > group:
        w[:group] = 0  # a group of zeros
    got = ds4a.rmsnorm_fp8(up(torch, x), up(torch, w), eps=1e-6, residual=up(torch, r), group=group, want_y=True)
    codes, scales = host(got[0]), host(got[1])
    h, y = paged.rmsnorm(x, w, 1e-6, r)
    if residual:
        assert np.array_equal(host(got[2]), (x.astype(np.float32) + r.astype(np.float32)).astype(dt))
    assert (np.abs(host(got[-1]).astype(np.float64) - y) <= np.abs(y) * (F16 + 2.0 ** -18) + 2.0 ** -25).all()
    want_s = paged.group_scales(y, group)
    assert (np.abs(scales - want_s) <= want_s * 2.0 ** -18).all()
    z = y / np.maximum(np.repeat(want_s, group or width, axis=1)[:, :width], 1e-300)
    off = np.abs(fp8.decode_table()[codes] - z)
    assert (off <= 0.5 * paged.e4m3_step(z) * (1 + 1e-9) + np.abs(z) * 2.0 ** -17).all()


@pytest.mark.parametrize("size", [1e-36, 1e-25, 1e-12, 1e12, 1e18])
def test_norm_of_rows_of_any_size(torch, ds4a, size):
    """fp32 rows from 1e-36 to 1e12, and one tiny group beside ordinary ones; rows of zeros; rows of 1e18, whose
    squares add up to more than fp32 holds (512e36 > 3.4e38), have y = 0."""
    rng = np.random.default_rng(72)
    x = (rng.standard_normal((3, 512)) * size).astype(np.float32)
    x[1] = 0
    x[2, :128] *= np.float32(1e-6)
    w = np.ones(512, dtype=np.float32)
    codes, scales, y = ds4a.rmsnorm_fp8(up(torch, x), up(torch, w), eps=1e-37, group=128, want_y=True)
    _, want = paged.rmsnorm(x, w, 1e-37)
    with np.errstate(over="ignore"):
        want[np.isinf(np.square(x).sum(1))] = 0
    want_s = paged.group_scales(want, 128)
    got_s = host(scales)
    keep = want_s * 448 >= 2.0 ** -100
    assert (np.abs(got_s - want_s) <= want_s * 2.0 ** -18)[keep].all() and (got_s[1] == 0).all()
    z = want / np.maximum(np.repeat(want_s, 128, axis=1), 1e-300)
    off = np.abs(fp8.decode_table()[host(codes)] - z)
    ok = off <= 0.5 * paged.e4m3_step(z) * (1 + 1e-9) + np.abs(z) * 2.0 ** -17
    assert ok[np.repeat(keep, 128, axis=1)].all() and (host(codes)[got_s.max(1) == 0] == 0).all()


def test_norm_strides_in_place_and_parts(torch, ds4a):
    """Residual updated in place in padded rows; codes alone, y alone; the rows behind are left."""
    rng = np.random.default_rng(70)
    n, width = 6, 1032
    x, r = (rng.standard_normal((n, width)).astype(np.float16) for _ in range(2))
    w = np.ones(width, dtype=np.float32)
    big = torch.full((n + 2, width + 24), 9.0, dtype=torch.float16, device="cuda")
    big[:n, :width] = up(torch, r)
    codes = torch.full((n + 1, width + 8), 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((n + 1, 12), 2.0, device="cuda")
    ds4a.rmsnorm_fp8(up(torch, x), up(torch, w), residual=big[:n, :width], residual_out=big[:n, :width], group=128,
                     codes=codes[:n, :width], scales=scales[:n, :9])
    want = ds4a.rmsnorm_fp8(up(torch, x), up(torch, w), residual=up(torch, r), group=128)
    assert torch.equal(codes[:n, :width], want[0]) and torch.equal(scales[:n, :9], want[1])
    assert torch.equal(big[:n, :width], want[2])
    assert (big[n:] == 9).all() and (big[:, width:] == 9).all()
    assert (codes[n:] == 3).all() and (codes[:, width:] == 3).all()
    assert (scales[n:] == 2).all() and (scales[:, 9:] == 2).all()
    y = torch.empty((n, width), dtype=torch.float16, device="cuda")
    ds4a.prepare_rmsnorm_fp8(up(torch, x), up(torch, w), y=y)()
    _, wy = paged.rmsnorm(x, w, 1e-6)
    assert (np.abs(host(y) - wy) <= np.abs(wy) * (F16 + 2.0 ** -18) + 2.0 ** -25).all()


def test_norm_then_quantise_is_the_row_format(torch, ds4a):
    """Codes and scales of a normed row are those ds4a_quantize_kv_fp8 gives for fp16 values that need no rounding."""
    x = torch.zeros((4, 512), dtype=torch.float16, device="cuda")
    x[:, ::2] = torch.randint(-64, 64, (4, 256), device="cuda").half() / 64
    x[:, 0] = 1.0
    x[:, 1] = 0.0
    one = torch.ones(512, device="cuda")
    codes, scales, y = ds4a.rmsnorm_fp8(x, one, want_y=True)
    c2, s2 = ds4a.quantize_kv_fp8(y)
    # the norm quantises its fp32 values, the row call their fp16 roundings
    near = (scales[:, 0] - s2).abs() <= s2 * 2.0 ** -10
    assert near.all() and (codes != c2).float().mean() < 0.05


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("recorded", [False, True])
@pytest.mark.parametrize("f8", [False, True])
def test_serving_steps(torch, ds4a, f8, recorded):
    """Six steps of three sequences held at a budget: the new compressed row is normed, appended, attended
    to, weighed, and the weakest row evicted, all on a side stream; direct calls, or one recording replayed."""
    rng = np.random.default_rng(80 + f8)
    page, budget, ratio, n = 8, 40, 4, 3
    rows = [budget, budget, 25]
    seg = make(rng, n, [budget + page] * n, page, f8, True)
    dev = rows_on(torch, ds4a, seg)
    cap = paged.capacity(seg)
    shape = shape_of(ratio)
    stream = torch.cuda.Stream()
    w = rng.random((n, cap)).astype(np.float32)
    ids = np.tile(np.arange(cap, dtype=np.int32), (n, 1))
    geom = np.array([(r * ratio, 0, 0, r) for r in rows], dtype=np.int32)
    d = dict(w=up(torch, w), ids=up(torch, ids), geom=up(torch, geom), q=torch.zeros((n, H, D), device="cuda").half(),
             x=torch.zeros((n, D), device="cuda").half(), slots=torch.zeros(n, dtype=torch.int32, device="cuda"),
             y=torch.zeros((n, D), device="cuda").half(), o=torch.zeros((n, H, D), device="cuda").half(),
             lse=torch.zeros((n, H), device="cuda"), kept=torch.zeros((n, budget), dtype=torch.int32, device="cuda"))
    gain = up(torch, (1 + 0.1 * rng.standard_normal(D)).astype(np.float32))
    ws = torch.empty(ds4a.decode_paged_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    we = torch.empty(ds4a.evict_paged_workspace_bytes(n, budget), dtype=torch.uint8, device="cuda")

    def calls():
        ds4a.prepare_rmsnorm_fp8(d["x"], gain, y=d["y"], stream=stream)()
        ds4a.append_paged(dev, d["y"], None, d["slots"], stream=stream)
        ds4a.attn_decode_paged(shape, d["geom"], d["q"], None, dev, workspace=ws, out=d["o"], lse=d["lse"],
                               stream=stream)
        ds4a.attn_weights_paged(shape, d["geom"], d["q"], dev, d["lse"], weights=d["w"], decay=0.9, out=d["w"],
                                stream=stream)
        ds4a.evict_paged(shape, d["geom"], dev, d["w"], budget, n_first=2, n_recent=5, ids=d["ids"], kept=d["kept"],
                         n_out=d["geom"][:, 3], workspace=we, stream=stream)

    torch.cuda.synchronize()
    graph = None
    if recorded:
        with ds4a.Graph(stream) as graph:
            calls()
    for step in range(6):
        geom[:, 0] += ratio
        at = geom[:, 3].copy()
        geom[:, 3] += 1
        x = rng.standard_normal((n, D)).astype(np.float16)
        q = rng.standard_normal((n, H, D)).astype(np.float16)
        slots = seg["table"][np.arange(n), at // page] * page + at % page
        new_id = geom[:, 0] // ratio - 1
        for b in range(n):
            ids[b, at[b]] = new_id[b]
            w[b, at[b]] = 0
        for name, val in (("geom", geom), ("x", x), ("q", q), ("slots", slots.astype(np.int32)), ("ids", ids), ("w", w)):
            d[name].copy_(up(torch, val))
        torch.cuda.synchronize()
        graph() if recorded else calls()
        torch.cuda.synchronize()
        # the oracle takes the device's normed rows as its new rows
        y = host(d["y"])
        for b in range(n):
            to = (int(seg["table"][b, at[b] // page]), int(at[b] % page))
            if f8:
                c, s = fp8.quantize_rows(y[b:b + 1])
                seg["k"][to], seg["k_scale"][to] = c[0], s[0]
            else:
                seg["k"][to] = y[b]
        check_decode(host(d["o"]), host(d["lse"]), paged.decode(shape, geom, q, None, seg), [cap] * n)
        after = paged.weights(shape, geom, q, seg, host(d["lse"]), w, 0.9)
        kept = host(d["kept"])
        got_n = host(d["geom"])[:, 3]
        for b in range(n):
            no, kp = got_n[b], kept[b, :got_n[b]]
            assert no == min(geom[b, 3], budget)
            got = host(d["w"])[b, :no]
            np.testing.assert_allclose(got, after[b][kp], rtol=1e-4)
            # the device's own weights (before the eviction: those now in kept slots, and the lost ones below) rank
            lost = [j for j in range(geom[b, 3]) if j not in set(kp)]
            safe = {j for j in range(geom[b, 3]) if ids[b, j] < 2 or ids[b, j] >= (geom[b, 0] + 1) // ratio - 5}
            assert not safe & set(lost)
            for j in lost:
                assert after[b][j] <= min(after[b][i] for i in kp if i not in safe) * (1 + 1e-4)
            ids[b, :no] = ids[b][kp]
            assert np.array_equal(host(d["ids"])[b, :no], ids[b, :no])
            w[b] = host(d["w"])[b]
            paged.move_rows(seg, b, kp)
            geom[b, 3] = no
        assert np.array_equal(host(dev.k).view(np.uint8), seg["k"].view(np.uint8))
    if graph is not None:
        graph.close()


def test_the_documented_serving_step(torch, ds4a):
    """The README's paged cache and its step, run as they stand: three steps of two sequences at the budget.  A row
    appended after an eviction starts from weight 0 and not from what its slot's last row received."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (setup,), (step,) = [b for b in blocks if "PagedRows(" in b], [b for b in blocks if "append_paged(" in b]
    rng = np.random.default_rng(95)
    n, budget, ratio = 2, 1024, 4
    pages = budget // 64 + 1
    pos = budget * ratio + 1
    tables = rng.permutation(1024)[:n * pages].reshape(n, pages).astype(np.int32)
    raw_rows = rng.standard_normal((4 * n, 64, D)).astype(np.float16)
    names = dict(torch=torch, ds4a=ds4a, n_seq=n, comp_table=up(torch, tables), raw_pool=up(torch, raw_rows),
                 raw_table=up(torch, np.arange(4 * n, dtype=np.int32).reshape(n, 4)), q_pos=pos, n_raw=192,
                 raw_pos0=pos - 191, n_comp=budget)
    exec(setup, names)
    names["pool"].copy_(up(torch, rng.standard_normal((1024, 64, D)).astype(np.float16)))
    for i in range(1, 4):
        q, new = rng.standard_normal((n, H, D)).astype(np.float16), rng.standard_normal((n, D)).astype(np.float16)
        names["geom"][:, 0], names["geom"][:, 2] = pos + ratio * i, pos + ratio * i - 191
        names.update(q=up(torch, q), new_k=up(torch, new), new_ids=budget + i - 1)
        w, ids = host(names["weights"]).copy(), host(names["ids"]).copy()
        geom = host(names["geom"]).copy()
        k = host(names["pool"]).copy()
        exec(step, names)
        assert (geom[:, 3] == budget).all() and (host(names["geom"])[:, 3] == budget).all()
        w[:, budget], ids[:, budget] = 0, budget + i - 1
        k[tables[:, budget // 64], budget % 64] = new
        geom[:, 3] += 1
        comp, raw = dict(k=k, v=k, table=tables), dict(k=raw_rows, v=raw_rows, table=host(names["raw_table"]))
        shape = shape_of(ratio)
        want = paged.decode(shape, geom, q, raw, comp)
        check_decode(host(names["o"]), host(names["lse"]), want, [budget + 129] * n)
        after = paged.weights(shape, geom, q, comp, host(names["lse"]), w, 1.0)
        got_w, got_ids = host(names["weights"]), host(names["ids"])
        for b in range(n):
            weight = dict(zip(ids[b, :budget + 1].tolist(), after[b, :budget + 1]))
            left = got_ids[b, :budget].tolist()
            assert len(set(left)) == budget and set(left) < set(weight) and budget + i - 1 in left
            # a score is off by 512 * 2^-23 of scale sum |q||k|, 17 here: 1.04e-3 of a weight
            np.testing.assert_allclose(got_w[b, :budget], [weight[x] for x in left], rtol=2e-3)


def test_two_streams_at_once(torch, ds4a):
    """Two decode steps in flight on two streams with their own workspaces."""
    rng = np.random.default_rng(90)
    shape = shape_of()
    jobs = []
    for k in range(2):
        geom, q, raw, comp = case(rng, [900, 40 + k], 4, 16, bool(k), True)
        jobs.append((geom, q, raw, comp, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                     rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = [ds4a.attn_decode_paged(shape, j[4], j[5], j[6], j[7], want_lse=True, stream=j[8],
                                       workspace=torch.empty(ds4a.decode_paged_workspace_bytes(2), dtype=torch.uint8,
                                                             device="cuda"),
                                       out=torch.empty_like(j[5]), lse=torch.empty((2, H), device="cuda"))
                for j in jobs]
        torch.cuda.synchronize()
    for (geom, q, raw, comp, *_), (o, lse) in zip(jobs, outs):
        check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [1028, 170])


def test_two_streams_without_workspaces_of_the_callers(torch, ds4a):
    """Decodes in flight on two streams, their outputs and workspaces made by the calls, nothing waited for between
    them: each call has its own, and a job's results are the same bits every time."""
    rng = np.random.default_rng(93)
    shape = shape_of()
    jobs = []
    for k in range(2):
        geom, q, raw, comp = case(rng, [4000 + k, 2500], 4, 16, bool(k), True)
        jobs.append((geom, q, raw, comp, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                     rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[ds4a.attn_decode_paged(shape, j[4], j[5], j[6], j[7], want_lse=True, stream=j[8]) for j in jobs]
            for _ in range(20)]
    torch.cuda.synchronize()
    for k, (geom, q, raw, comp, *_) in enumerate(jobs):
        check_decode(host(outs[0][k][0]), host(outs[0][k][1]), paged.decode(shape, geom, q, raw, comp), [4129, 2628])
        for o in outs[1:]:
            assert torch.equal(o[k][0], outs[0][k][0]) and torch.equal(o[k][1], outs[0][k][1])


def test_two_streams_with_workspaces_held(torch, ds4a):
    """The same with a workspace each that lives as long as the calls use it."""
    rng = np.random.default_rng(94)
    shape = shape_of()
    jobs = []
    for k in range(2):
        geom, q, raw, comp = case(rng, [3000, 800 + k], 4, 16, bool(k), True)
        o, lse = torch.empty((2, H, D), dtype=torch.float16, device="cuda"), torch.empty((2, H), device="cuda")
        ws = torch.empty(ds4a.decode_paged_workspace_bytes(2), dtype=torch.uint8, device="cuda")
        call = ds4a.prepare_decode_paged(shape, up(torch, np.array(geom, dtype=np.int32)), up(torch, q),
                                         rows_on(torch, ds4a, raw), rows_on(torch, ds4a, comp), workspace=ws, out=o,
                                         lse=lse, stream=torch.cuda.Stream())
        jobs.append((geom, q, raw, comp, o, lse, call))
    assert jobs[0][6]._keep[6].data_ptr() != jobs[1][6]._keep[6].data_ptr()
    torch.cuda.synchronize()
    for _ in range(50):
        for j in jobs:
            j[6]()
    torch.cuda.synchronize()
    for geom, q, raw, comp, o, lse, _ in jobs:
        check_decode(host(o), host(lse), paged.decode(shape, geom, q, raw, comp), [3128, 930])


def test_weights_on_a_side_stream_while_the_current_one_is_busy(torch, ds4a):
    """The output made by the call is zeroed on the call's stream, before its kernel, not when the current stream
    gets to it."""
    rng = np.random.default_rng(92)
    rows = [300, 77]
    geom = geometry(rows, 4, 16)
    comp = make(rng, 2, rows, 16)
    shape, g, q, seg = shape_of(), up(torch, np.array(geom, dtype=np.int32)), up(torch, rng.standard_normal(
        (2, H, D)).astype(np.float16)), rows_on(torch, ds4a, comp)
    _, lse = ds4a.attn_decode_paged(shape, g, q, None, seg, want_lse=True)
    want = ds4a.attn_weights_paged(shape, g, q, seg, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # some 10 ms of the current stream
    got = ds4a.attn_weights_paged(shape, g, q, seg, lse, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and got.sum() > 100


def test_a_bad_call_records_nothing(torch, ds4a):
    rng = np.random.default_rng(91)
    seg = make(rng, 1, [20], 4)
    dev = rows_on(torch, ds4a, seg)
    g = torch.tensor([[100, 0, 0, 20]], dtype=torch.int32, device="cuda")
    q = torch.zeros((1, H, D), dtype=torch.float16, device="cuda")
    with pytest.raises(ds4a.Ds4aError) as e:
        ds4a.attn_decode_paged(shape_of(), g, q, None, dev, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ds4a.ERR_WORKSPACE
    torch.cuda.synchronize()
