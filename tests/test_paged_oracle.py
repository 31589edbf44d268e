"""The paged-cache oracle against the layout oracle, the definition by lists, and hand-made cases (CPU)."""

import numpy as np
import pytest

import oracle
from oracle import fp8, paged

D = 512


def make(rng, n_seq, rows, page, fp8_rows=False, shared=False, absent=()):
    """A segment whose pages lie in random order in the pool."""
    per = [-(-r // page) for r in rows]
    order = rng.permutation(max(sum(per), 1))
    table = np.full((n_seq, max(max(per), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    for b, i in absent:
        table[b, i] = len(order) + 3
    k = rng.standard_normal((len(order), page, D)).astype(np.float16)
    v = k if shared else rng.standard_normal(k.shape).astype(np.float16)
    seg = dict(k=k, v=v, table=table)
    if fp8_rows:
        for name in ("k",) if shared else ("k", "v"):
            c, s = fp8.quantize_rows(seg[name].reshape(-1, D))
            seg[name], seg[name + "_scale"] = c.reshape(k.shape), s.reshape(k.shape[:2])
        if shared:
            seg["v"], seg["v_scale"] = seg["k"], seg["k_scale"]
    return seg


SHAPE = dict(ratio=4, window=128, scale=1.0 / np.sqrt(512.0))


def test_decode_is_the_layout_oracle_on_gathered_rows():
    rng = np.random.default_rng(1)
    rows, pos = [0, 1, 77, 300], [130, 4, 311, 1300]
    comp = make(rng, 4, rows, 16)
    raw = make(rng, 4, [131, 5, 200, 140], 24)
    geom = [(pos[0], 131, 0, 0), (pos[1], 5, 0, 1), (pos[2], 200, 112, 77), (pos[3], 140, 1161, 300)]
    q = rng.standard_normal((4, 64, D)).astype(np.float16)
    o, lse, _, _ = paged.decode(SHAPE, geom, q, raw, comp)
    for b, (p, nr, r0, nc) in enumerate(geom):
        L = dict(T=1, q_pos0=p, n_raw=nr, raw_pos0=r0, n_comp=nc, **SHAPE)
        rows_of = [paged.segment_rows(s, b, n, w)[0].astype(np.float16)
                   for s, n in ((raw, nr), (comp, nc)) for w in ("k", "v")]
        want, want_l = oracle.attention(L, q[b:b + 1], *rows_of)
        np.testing.assert_allclose(o[b], want[0], rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[b], want_l[0], rtol=0, atol=1e-12)


def test_weights_of_a_step_sum_to_the_heads():
    """Over rows all seen through the compressed segment the weights of a step
    sum to 64; an absent page's rows get none; rows beyond the geometry are not written."""
    rng = np.random.default_rng(2)
    comp = make(rng, 2, [50, 9], 8, absent=((0, 2),))
    geom = [(4 * 50, 0, 0, 50), (4 * 9, 0, 0, 9)]
    q = rng.standard_normal((2, 64, D)).astype(np.float16)
    _, lse, _, _ = paged.decode(SHAPE, geom, q, None, comp)
    w = paged.weights(SHAPE, geom, q, comp, lse, None, 1.0)
    np.testing.assert_allclose(np.nansum(w, 1), 64.0, rtol=1e-12)
    assert (w[0, 16:24] == 0).all() and np.isnan(w[1, 9:]).all() and np.isnan(w[0, 50:]).all()


@pytest.mark.parametrize("seed", range(4))
def test_evict_keeps_the_best_and_moves_the_fewest(seed):
    rng = np.random.default_rng(seed)
    n, keep = 40, 23
    w = rng.integers(0, 6, (1, n)).astype(np.float32)
    w[0, 3] = np.nan
    ids = rng.permutation(n)[None].astype(np.int32)
    (n_out, kept), = paged.evict(SHAPE, [(4 * n, 0, 0, n)], w, ids, keep, 2, 5, n)
    assert n_out == keep and len(set(kept)) == keep
    safe = {j for j in range(n) if ids[0, j] < 2 or ids[0, j] >= n - 5}
    assert safe <= set(kept)
    gone = sorted(set(range(n)) - set(kept))
    worst = min((w[0, j], -j) for j in kept if j not in safe)
    assert all(np.isnan(w[0, j]) or (w[0, j], -j) < worst for j in gone)
    assert all(kept[i] == i or i in gone for i in range(keep))
    moved = [j for i, j in enumerate(kept) if i != j]
    assert moved == sorted(moved) and all(j >= keep for j in moved)


def test_rmsnorm_by_hand():
    x = np.array([[3.0, 4.0] + [0.0] * 6], dtype=np.float32)
    h, y = paged.rmsnorm(x, np.full(8, 2.0, dtype=np.float32), 1e-30)
    np.testing.assert_allclose(y[0, :2], np.array([3.0, 4.0]) / np.sqrt(25 / 8) * 2, rtol=1e-12)
    np.testing.assert_allclose(paged.group_scales(y, 0), [[y[0, 1] / 448]], rtol=1e-15)
    assert paged.e4m3_step(np.array([448.0, 1.0, 1.99, 2.0 ** -6, 1e-4])).tolist() == \
        [32.0, 0.125, 0.125, 2.0 ** -9, 2.0 ** -9]
