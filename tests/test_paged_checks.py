"""Refusals of the paged cache calls and of the norm, without a GPU: the C ABI
rejects bad arguments before touching CUDA (an unsupported device or a CUDA
error is what a call with good ones answers here), and the binding rejects
tensors that do not fit."""

import concurrent.futures as cf
import ctypes
import math
import os
import re

import pytest
import torch

from mqa_flash_attention_gb300 import build as ds4a_build
from mqa_flash_attention_gb300 import ds4a

H, D = 64, 512
F16, F32, I32, U8 = torch.float16, torch.float32, torch.int32, torch.uint8
AT = 1 << 24  # never dereferenced: host checks only
SHAPE = dict(T=1, q_pos0=0, n_raw=0, raw_pos0=0, n_comp=0, ratio=4, window=128)


@pytest.fixture(scope="module")
def lib():
    ds4a_build.build()
    return ds4a.lib()


def seg(**kw):
    base = dict(k=AT, v=2 * AT, row_stride=1024, page_stride=16 * 1024, page_rows=16, n_pages=8, k_scale=None,
                v_scale=None, table=3 * AT, table_stride=32, max_pages=8)
    base.update(kw)
    return ds4a.PagedSegment(*[base[n] for n, _ in ds4a.PagedSegment._fields_])


def batch(raw=None, comp=None, **kw):
    base = dict(q=4 * AT, q_seq_stride=65536, o=5 * AT, o_seq_stride=65536, lse=6 * AT)
    base.update(kw)
    return ds4a.PagedBatch(base["q"], base["q_seq_stride"], raw if raw is not None else seg(),
                           comp if comp is not None else seg(), base["o"], base["o_seq_stride"], base["lse"])


def decode(lib, X, n=2, shape=None, geom=7 * AT, ws=1 << 30, nbytes=None):
    S = ds4a.make_layout(dict(SHAPE, **(shape or {})))
    need = lib.ds4a_attn_decode_paged_workspace_size(n)
    return elsewhere(lib.ds4a_attn_decode_paged, n, ctypes.byref(S), geom, ctypes.byref(X), ws,
                     need if nbytes is None else nbytes, None)


def elsewhere(fn, *args):
    """A call on a thread of its own: the CUDA error text is kept per thread."""
    with cf.ThreadPoolExecutor(1) as ex:
        return ex.submit(fn, *args).result()


def passes(status):
    """Past every check: what is left to fail here is the missing device."""
    return status in (ds4a.ERR_CUDA, ds4a.ERR_UNSUPPORTED)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are made up")


@needs_no_gpu
def test_good_decode_arguments_reach_the_device(lib):
    assert passes(decode(lib, batch()))
    assert passes(decode(lib, batch(raw=seg(max_pages=0, k=None), lse=None)))
    f8 = seg(row_stride=512, page_stride=8192, k_scale=AT, v_scale=AT)
    assert passes(decode(lib, batch(raw=f8, comp=f8)))
    assert passes(decode(lib, batch(comp=seg(page_rows=1, page_stride=1024))))
    assert decode(lib, batch(), n=0) == ds4a.OK


@needs_no_gpu
@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=AT + 8), dict(v=AT + 4), dict(row_stride=1008), dict(row_stride=1032),
    dict(page_stride=15 * 1024), dict(page_stride=16 * 1024 + 8), dict(page_rows=0), dict(n_pages=0),
    dict(table=None), dict(table=AT + 2), dict(table_stride=28), dict(table_stride=34), dict(max_pages=-1),
    dict(page_rows=1 << 28, page_stride=(1 << 39) - 16), dict(k_scale=AT), dict(v_scale=AT),
    dict(k_scale=AT, v_scale=AT),  # E4M3 beside an fp16 segment
    dict(row_stride=1 << 39, page_stride=(1 << 43))])
def test_bad_segments_are_refused(lib, bad):
    assert decode(lib, batch(comp=seg(**bad))) == ds4a.ERR_INVALID_ARG
    assert decode(lib, batch(raw=seg(**bad))) == ds4a.ERR_INVALID_ARG


@needs_no_gpu
@pytest.mark.parametrize("bad", [dict(q=None), dict(q=AT + 8), dict(q_seq_stride=65520), dict(o=None),
                                 dict(o_seq_stride=65544), dict(lse=AT + 2)])
def test_bad_batches_are_refused(lib, bad):
    assert decode(lib, batch(**bad)) == ds4a.ERR_INVALID_ARG


@needs_no_gpu
def test_bad_decode_calls_are_refused(lib):
    X = batch()
    assert decode(lib, X, n=-1) == ds4a.ERR_INVALID_ARG
    for shape in (dict(window=0), dict(ratio=0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38)):
        S = ds4a.make_layout(dict(SHAPE, **shape))
        S.ratio = shape.get("ratio", 4)
        assert lib.ds4a_attn_decode_paged(2, ctypes.byref(S), 7 * AT, ctypes.byref(X), AT, 1 << 40, None) == \
            ds4a.ERR_INVALID_ARG
    # The window's rows and the compressed ones together: 2^30 at most.
    most = seg(page_rows=1 << 27, n_pages=8, page_stride=1 << 37, table_stride=32, max_pages=8)
    assert decode(lib, batch(comp=most)) == ds4a.ERR_INVALID_ARG
    assert passes(decode(lib, batch(raw=seg(max_pages=0), comp=most)))
    assert decode(lib, X, geom=None) == ds4a.ERR_INVALID_ARG
    assert decode(lib, X, geom=AT + 4) == ds4a.ERR_INVALID_ARG
    assert decode(lib, X, ws=None) == ds4a.ERR_WORKSPACE
    assert decode(lib, X, ws=AT + 128) == ds4a.ERR_WORKSPACE
    assert decode(lib, X, nbytes=lib.ds4a_attn_decode_paged_workspace_size(2) - 1) == ds4a.ERR_WORKSPACE
    assert lib.ds4a_attn_decode_paged(2, None, 7 * AT, ctypes.byref(X), AT, 1 << 40, None) == ds4a.ERR_INVALID_ARG


def source_of(function):
    """The body of a __device__ function of paged_attn.cu, comments taken out."""
    with open(os.path.join(ds4a_build.CSRC, "paged_attn.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index(function + "(const PagedAttnParams &p")
    start, depth = text.index("{", at), 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(function)


@pytest.mark.parametrize("role", ["softmax_role", "weights_role"])
def test_compute_roles_vote_after_a_wait(role):
    """A wait may run out in some threads of a block and not in others.  What follows it and needs all
    threads (a plain barrier), or depends on what was waited for (addresses), comes after a vote."""
    voted, seen = True, set()
    for m in re.finditer(r"mbar_wait\(|bar_red_or\(|bar_sync_id\(|p\.(?:acc_in|lse_in|acc_out|lse|ws_ml)\[", source_of(role)):
        seen.add(m.group())
        if m.group() == "mbar_wait(":
            voted = False
        elif m.group() == "bar_red_or(":
            voted = True
        else:
            assert voted, f"{role}: {m.group()} after a wait without a vote"
    assert {"mbar_wait(", "bar_red_or(", "bar_sync_id("} <= seen and voted


def test_plan_counts_lie_where_no_bulk_copy_writes():
    """Block-wide plans store counts with ordinary stores; a TMA copy into the same bytes is not ordered after
    them by a block barrier, so they stay out of what TMA fills (Q and the K/V ring)."""
    with open(os.path.join(ds4a_build.CSRC, "paged_attn.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.findall(r"plan_block<WEIGHTS>\(p, ms, reinterpret_cast<int \*>\(smem \+ (\w+)\)\)", text)
    filled = set(re.findall(r"tma_load_4d\(sbase \+ (\w+)", text)) | \
        set(re.findall(r"const uint32_t stage = sbase \+ (\w+)", text))
    assert filled == {"kOffQ", "kOffKV"} and at == ["kOffP"]


def weights(lib, X=None, acc=8 * AT, acc_stride=512, decay=1.0, out=9 * AT, out_stride=512, n=2):
    S = ds4a.make_layout(SHAPE)
    return elsewhere(lib.ds4a_attn_weights_paged, n, ctypes.byref(S), 7 * AT, ctypes.byref(X or batch()), acc,
                     acc_stride, decay, out, out_stride, None)


@needs_no_gpu
def test_weights_arguments_are_checked(lib):
    assert passes(weights(lib))
    assert passes(weights(lib, acc=None, acc_stride=0))
    assert passes(weights(lib, acc=9 * AT))
    assert passes(weights(lib, batch(comp=seg(v=None), raw=seg(k=None), o=None)))
    for bad in (dict(acc_stride=508), dict(acc=AT + 2), dict(out=None), dict(out=AT + 1), dict(out_stride=500),
                dict(decay=math.nan), dict(decay=math.inf), dict(acc=9 * AT + 512), dict(acc=9 * AT, acc_stride=516),
                dict(X=batch(lse=None)), dict(X=batch(q=None)), dict(X=batch(comp=seg(k=None))), dict(n=-1)):
        assert weights(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    assert weights(lib, batch(comp=seg(max_pages=0))) == ds4a.OK


def evict(lib, rows=None, n=2, keep=100, first=0, recent=0, w=8 * AT, ws=512, ids=None, ids_stride=0, kept=9 * AT,
          kept_stride=400, wo=None, wo_stride=0, io=None, io_stride=0, n_out=10 * AT, no_stride=4, work=1 << 30,
          nbytes=1 << 20, geom=7 * AT):
    S = ds4a.make_layout(SHAPE)
    E = ds4a.Eviction(w, ws, ids, ids_stride, keep, first, recent, kept, kept_stride, wo, wo_stride, io, io_stride,
                      n_out, no_stride)
    return elsewhere(lib.ds4a_evict_paged, n, ctypes.byref(S), geom, ctypes.byref(rows or seg()), ctypes.byref(E), work,
                     nbytes, None)


@needs_no_gpu
def test_evict_arguments_are_checked(lib):
    assert passes(evict(lib))
    assert passes(evict(lib, wo=8 * AT, wo_stride=512, ids=11 * AT, ids_stride=512, io=11 * AT, io_stride=512,
                        no_stride=16))
    for bad in (dict(keep=0), dict(first=-1), dict(recent=-1), dict(w=None), dict(ws=508), dict(w=AT + 2),
                dict(kept=None), dict(kept_stride=396), dict(kept=AT + 1), dict(n_out=None), dict(no_stride=2),
                dict(n_out=AT + 2), dict(ids=AT, ids_stride=512), dict(io=AT, io_stride=512),
                dict(wo=8 * AT + 4, wo_stride=512), dict(wo=8 * AT, wo_stride=516), dict(wo=12 * AT, wo_stride=4),
                dict(ids=AT, ids_stride=512, io=AT, io_stride=1024), dict(geom=None), dict(geom=AT + 8), dict(n=-1),
                dict(rows=seg(max_pages=0)), dict(rows=seg(table=None)), dict(rows=seg(v=None))):
        assert evict(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    need = lib.ds4a_evict_paged_workspace_size(2, 100)
    assert need >= 4 * 2 + 8 * 2 * 100
    for bad in (dict(work=None), dict(work=AT + 64), dict(nbytes=need - 1)):
        assert evict(lib, **bad) == ds4a.ERR_WORKSPACE, bad
    assert evict(lib, n=0) == ds4a.OK
    assert lib.ds4a_evict_paged_workspace_size(0, 4) == 0


def append(lib, rows=None, n=4, k=8 * AT, v=9 * AT, stride=1024, slots=10 * AT):
    return elsewhere(lib.ds4a_append_paged, ctypes.byref(rows or seg()), n, k, v, stride, slots, None)


@needs_no_gpu
def test_append_arguments_are_checked(lib):
    assert passes(append(lib))
    assert passes(append(lib, seg(v=AT), v=None))
    assert passes(append(lib, seg(table=None, max_pages=0)))
    for bad in (dict(k=None), dict(v=None), dict(k=AT * 8 + 8), dict(stride=1000), dict(stride=512), dict(slots=None),
                dict(slots=AT + 2), dict(n=-1), dict(k=AT), dict(v=AT + 1024), dict(rows=seg(k=None)),
                dict(rows=seg(page_rows=0)), dict(k=2 * AT + 16 * 1024 * 8 - 1024)):
        assert append(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    assert append(lib, n=0) == ds4a.OK


@needs_no_gpu
def test_append_refuses_one_scale_for_two_rows(lib):
    """K and V rows apart need a scale array each (4 * 16 scales a page, 8 pages: 512 bytes)."""
    f8 = dict(row_stride=512, page_stride=8192)
    assert passes(append(lib, seg(k_scale=11 * AT, v_scale=12 * AT, **f8)))
    assert passes(append(lib, seg(k_scale=11 * AT, v_scale=11 * AT + 512, **f8)))
    assert passes(append(lib, seg(v=AT, k_scale=11 * AT, v_scale=11 * AT, **f8), v=None))
    assert passes(append(lib, seg(v=AT, k_scale=11 * AT, v_scale=12 * AT, **f8), v=None))
    for bad in (seg(k_scale=11 * AT, v_scale=11 * AT, **f8), seg(k_scale=11 * AT, v_scale=11 * AT + 508, **f8),
                seg(v=AT, k_scale=11 * AT, v_scale=11 * AT + 4, **f8)):
        assert append(lib, bad) == ds4a.ERR_INVALID_ARG


def norm(lib, n=3, width=64, f32=0, x=AT, xs=128, r=None, rs=0, ro=None, ros=0, w=2 * AT, eps=1e-6, group=0, c=3 * AT,
         cs=64, s=4 * AT, ss=4, y=None, ys=0):
    N = ds4a.Norm(n, width, f32, group, x, xs, r, rs, ro, ros, w, eps, c, cs, s, ss, y, ys)
    return elsewhere(lib.ds4a_rmsnorm_fp8, ctypes.byref(N), None)


@needs_no_gpu
def test_norm_arguments_are_checked(lib):
    assert passes(norm(lib))
    assert passes(norm(lib, r=5 * AT, rs=128, ro=5 * AT, ros=128))
    assert passes(norm(lib, r=5 * AT, rs=128, ro=AT, ros=128))
    assert passes(norm(lib, c=None, s=None, y=6 * AT, ys=128))
    assert passes(norm(lib, group=32, ss=8))
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(width=4), dict(width=60), dict(width=32776, xs=1 << 17, cs=32776), dict(group=16),
                dict(group=-32), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e-40),
                dict(x=None), dict(x=AT + 8), dict(xs=120), dict(xs=136), dict(f32=1), dict(w=None), dict(w=AT + 4),
                dict(r=5 * AT, rs=128), dict(ro=5 * AT, ros=128), dict(r=5 * AT, rs=128, ro=5 * AT + 16, ros=128),
                dict(r=5 * AT, rs=128, ro=5 * AT, ros=256), dict(c=None), dict(s=None), dict(c=None, s=None),
                dict(c=AT + 4), dict(cs=60), dict(cs=68), dict(group=32, ss=4), dict(s=AT + 2), dict(y=AT + 8, ys=128),
                dict(y=6 * AT, ys=64), dict(c=AT), dict(y=3 * AT, ys=128), dict(s=3 * AT + 8)):
        assert norm(lib, **bad) == ds4a.ERR_INVALID_ARG, bad
    assert norm(lib, n=0) == ds4a.OK


# ------------------------------------------------------------------ binding

def raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_paged_rows_refuses_what_does_not_fit():
    k = torch.zeros((4, 8, D), dtype=F16)
    c, s = torch.zeros((4, 8, D), dtype=U8), torch.zeros((4, 8))
    t = torch.zeros((2, 3), dtype=I32)
    raises("fp16", ds4a.PagedRows, k.float(), None, t)
    raises("fp16", ds4a.PagedRows, c, None, t)
    raises("uint8", ds4a.PagedRows, k, None, t, k_scale=s)
    raises("n_pages", ds4a.PagedRows, k[:, :, :256], None, t)
    raises("contiguous rows", ds4a.PagedRows, k.transpose(1, 2).contiguous().transpose(1, 2), None, t)
    raises("share shape", ds4a.PagedRows, k, k[:, :4].clone(), t)
    raises("share shape", ds4a.PagedRows, k, torch.zeros((4, 9, D), dtype=F16)[:, :8], t)
    raises("k_scale", ds4a.PagedRows, c, None, t, k_scale=s[:3])
    raises("v_scale", ds4a.PagedRows, c, c.clone(), t, k_scale=s)
    raises("k_scale", ds4a.PagedRows, c, c.clone(), t, v_scale=s)
    raises("table", ds4a.PagedRows, k, None, t.long())
    raises("table", ds4a.PagedRows, k, None, t.t())
    r = ds4a.PagedRows(c, None, t, k_scale=s)
    assert r.v is c and r.v_scale is s and r.capacity == 24


def test_paged_calls_refuse_what_does_not_fit():
    rows = ds4a.PagedRows(torch.zeros((4, 8, D), dtype=F16), None, torch.zeros((2, 3), dtype=I32))
    q, geom = torch.zeros((2, H, D), dtype=F16), torch.zeros((2, 4), dtype=I32)
    raises("CUDA", ds4a.attn_decode_paged, SHAPE, geom, q, None, rows)
    raises("q must be", ds4a.attn_decode_paged, SHAPE, geom, q.float(), None, rows)
    raises("out has", ds4a.attn_decode_paged, SHAPE, geom, q, None, rows, out=torch.zeros((3, H, D), dtype=F16))
    raises("lse must be", ds4a.attn_decode_paged, SHAPE, geom, q, None, rows, lse=torch.zeros((2, 63)))
    raises("lse", ds4a.attn_weights_paged, SHAPE, geom, q, rows, None)
    raises("CUDA", ds4a.append_paged, rows, torch.zeros((2, D), dtype=F16), None, torch.zeros(2, dtype=I32))
    raises("fp16 or fp32", ds4a.prepare_rmsnorm_fp8, torch.zeros((2, 8), dtype=torch.bfloat16), torch.ones(8))


@pytest.mark.parametrize("call", ["geom", "table", "no_table", "weights", "kept", "ids", "n_out", "slots", "v", "scales",
                                  "codes", "weight", "residual"])
def test_sizes_are_refused_before_devices(call, monkeypatch):
    """The size checks, with the device check taken away."""
    monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
    monkeypatch.setattr(ds4a, "_stream", lambda s: ctypes.c_void_p(0))
    pool = torch.zeros((4, 8, D), dtype=F16)
    rows = ds4a.PagedRows(pool, None, torch.zeros((2, 3), dtype=I32))
    q, geom, w = torch.zeros((2, H, D), dtype=F16), torch.zeros((2, 4), dtype=I32), torch.zeros((2, 24))
    lse, kept, n_out = torch.zeros((2, H)), torch.zeros((2, 10), dtype=I32), torch.zeros(2, dtype=I32)
    ev = lambda **kw: ds4a.prepare_evict_paged(SHAPE, geom, rows, kw.pop("weights", w), 10,  # noqa: E731
                                               **dict(dict(kept=kept, n_out=n_out), **kw))
    x, one = torch.zeros((2, 64), dtype=F16), torch.ones(64)
    if call == "geom":
        raises("seq_geom", ds4a.attn_decode_paged, SHAPE, geom[:1], q, None, rows)
        raises("seq_geom", ds4a.attn_decode_paged, SHAPE, geom.long(), q, None, rows)
    elif call == "table":
        short = ds4a.PagedRows(pool, None, torch.zeros((1, 3), dtype=I32))
        raises("table has 1", ds4a.attn_decode_paged, SHAPE, geom, q, None, short)
        raises("repeat", ds4a.attn_decode_paged, SHAPE, geom, q, None,
               ds4a.PagedRows(pool, None, torch.zeros((1, 3), dtype=I32).expand(2, 3)))
    elif call == "no_table":
        raises("no page table", ds4a.attn_weights_paged, SHAPE, geom, q, ds4a.PagedRows(pool), lse,
               out=torch.zeros((2, 0)))
    elif call == "weights":
        raises("weights must be", ds4a.attn_weights_paged, SHAPE, geom, q, rows, lse, weights=w[:, :23])
        raises("out must be", ds4a.attn_weights_paged, SHAPE, geom, q, rows, lse, out=w.double())
        raises("weights must be", ev, weights=w[:1])
    elif call == "kept":
        raises("kept must be", ev, kept=kept[:, :9])
    elif call == "ids":
        raises("go together", ev, ids=torch.zeros((2, 24), dtype=I32))
        raises("ids must be", ev, ids=torch.zeros((2, 23), dtype=I32), ids_out=torch.zeros((2, 24), dtype=I32))
    elif call == "n_out":
        raises("n_out", ev, n_out=n_out[:1])
    elif call == "slots":
        raises("slots", ds4a.append_paged, rows, torch.zeros((2, D), dtype=F16), None, torch.zeros(3, dtype=I32))
        raises("slots", ds4a.append_paged, rows, torch.zeros((2, D), dtype=F16), None, torch.zeros(2))
    elif call == "v":
        apart = ds4a.PagedRows(pool, pool.clone())
        raises("v is missing", ds4a.append_paged, apart, torch.zeros((2, D), dtype=F16), None, torch.zeros(2, dtype=I32))
    elif call == "scales":
        raises("scales", ds4a.rmsnorm_fp8, x, one, group=32, scales=torch.zeros((2, 1)))
    elif call == "codes":
        raises("codes", ds4a.rmsnorm_fp8, x, one, codes=torch.zeros((2, 63), dtype=U8))
    elif call == "weight":
        raises("weight", ds4a.rmsnorm_fp8, x, one.half())
    else:
        raises("residual", ds4a.rmsnorm_fp8, x, one, residual=x.float())


def test_rows_repeated_by_stride_are_refused(lib, monkeypatch):
    """One row expanded to several, or rows that overlap, are not read as rows of their own behind it."""
    monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
    monkeypatch.setattr(ds4a, "_stream", lambda s: ctypes.c_void_p(0))
    pool, slots = torch.zeros((4, 8, D), dtype=F16), torch.arange(3, dtype=I32)
    one, row = ds4a.PagedRows(pool), torch.zeros((1, D), dtype=F16)
    apart = ds4a.PagedRows(pool, torch.zeros_like(pool))
    for k in (row.expand(3, D), torch.zeros(4 * D, dtype=F16).as_strided((3, D), (256, 1))):
        for rows, v in ((one, None), (apart, k)):
            with pytest.raises(ds4a.Ds4aError) as e:
                elsewhere(ds4a.append_paged, rows, k, v, slots)
            assert e.value.status == ds4a.ERR_INVALID_ARG
    w, geom = torch.zeros((1, 24)), torch.zeros((3, 4), dtype=I32)
    rows = ds4a.PagedRows(pool, None, torch.zeros((3, 3), dtype=I32))
    q, lse = torch.zeros((3, H, D), dtype=F16), torch.zeros((3, H))
    raises("weights must be", ds4a.attn_weights_paged, SHAPE, geom, q, rows, lse, weights=w.expand(3, 24))
    raises("out must be", ds4a.attn_weights_paged, SHAPE, geom, q, rows, lse, out=w.expand(3, 24))
    raises("x must be", ds4a.rmsnorm_fp8, torch.zeros((1, 64), dtype=F16).expand(3, 64), torch.ones(64))
    with pytest.raises(ds4a.Ds4aError) as e:
        elsewhere(ds4a.attn_decode_paged, SHAPE, geom, q[:1].expand(3, H, D), None, rows)
    assert e.value.status == ds4a.ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["decode", "weights", "evict", "append", "norm", "norm_residual", "norm_y"])
def test_empty_batches_do_nothing(lib, call, monkeypatch):
    """No sequences, no rows: empty tensors have no address, and no call refuses them."""
    monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
    monkeypatch.setattr(ds4a, "_stream", lambda s: ctypes.c_void_p(0))
    rows = ds4a.PagedRows(torch.zeros((4, 8, D), dtype=F16), None, torch.zeros((0, 3), dtype=I32))
    q, geom, x = torch.zeros((0, H, D), dtype=F16), torch.zeros((0, 4), dtype=I32), torch.zeros((0, 64), dtype=F16)
    one = torch.ones(64)
    if call == "decode":
        o, lse = ds4a.attn_decode_paged(SHAPE, geom, q, rows, rows, want_lse=True)
        assert o.shape == (0, H, D) and lse.shape == (0, H)
    elif call == "weights":
        assert ds4a.attn_weights_paged(SHAPE, geom, q, rows, torch.zeros((0, H))).shape == (0, 24)
    elif call == "evict":
        kept, n_out = ds4a.evict_paged(SHAPE, geom, rows, torch.zeros((0, 24)), 10)
        assert kept.shape == (0, 10) and n_out.shape == (0,)
    elif call == "append":
        ds4a.append_paged(rows, torch.zeros((0, D), dtype=F16), None, torch.zeros(0, dtype=I32))
    elif call == "norm":
        codes, scales = ds4a.rmsnorm_fp8(x, one, group=32)
        assert codes.shape == (0, 64) and scales.shape == (0, 2)
    elif call == "norm_residual":
        assert ds4a.rmsnorm_fp8(x, one, residual=x)[2].shape == (0, 64)
    else:
        ds4a.prepare_rmsnorm_fp8(x, one, y=torch.zeros((0, 64), dtype=F16))()


# ------------------------------------------------------------------ streams

class Streams:
    """Stands in for torch's current stream: which stream was current at each allocation."""

    def __init__(self, monkeypatch):
        self.current, self.made = None, []
        outer = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, outer.current = outer.current, self.stream

            def __exit__(self, *exc):
                outer.current = self.before

        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(ds4a, "_on_device", lambda **kw: None)
        monkeypatch.setattr(ds4a, "_stream", lambda s: ctypes.c_void_p(0))
        for name in ("empty", "zeros", "empty_like"):
            def make(*a, real=getattr(torch, name), name=name, **kw):
                self.made.append((name, self.current))
                return real(*a, **kw)
            monkeypatch.setattr(torch, name, make)


class Library:
    """Every call succeeds; every size is 4096."""

    def __getattr__(self, name):
        return lambda *a: 4096 if "size" in name or "splits" in name else ds4a.OK


def test_weights_fill_their_output_on_the_stream_of_the_call(monkeypatch):
    rows = ds4a.PagedRows(torch.zeros((4, 8, D), dtype=F16), None, torch.zeros((2, 3), dtype=I32))
    q, geom, lse = torch.zeros((2, H, D), dtype=F16), torch.zeros((2, 4), dtype=I32), torch.zeros((2, H))
    monkeypatch.setattr(ds4a, "_lib", Library())
    s = Streams(monkeypatch)
    for stream in (None, "side"):
        s.made.clear()
        ds4a.attn_weights_paged(SHAPE, geom, q, rows, lse, stream=stream)
        assert s.made == [("zeros", stream)] and s.current is None


def wrapper_calls():
    """Every wrapper that makes tensors of its own, on small host tensors: (name, number of tensors, call)."""
    q, geom = torch.zeros((2, H, D), dtype=F16), torch.zeros((2, 4), dtype=I32)
    r, c, sc = torch.zeros((64, D), dtype=F16), torch.zeros((64, D), dtype=U8), torch.ones(64)
    b = torch.zeros((2, 64, D), dtype=F16)
    rows = ds4a.PagedRows(torch.zeros((4, 8, D), dtype=F16), None, torch.zeros((2, 3), dtype=I32))
    L = ds4a.make_layout(dict(T=2, q_pos0=100, n_raw=64, raw_pos0=38, n_comp=25, ratio=4, window=128))
    S = ds4a.make_layout(SHAPE)
    w, lse = torch.zeros((2, 24)), torch.zeros((2, H))
    x, one = torch.zeros((2, 64), dtype=F16), torch.ones(64)
    idx = torch.zeros((2, 8), dtype=I32)
    f8 = dict(k_comp_scale=sc, v_comp_scale=sc, k_raw_scale=sc, v_raw_scale=sc)
    kv, state = torch.zeros((5, 16)), torch.zeros((3, 16))
    qi, ki, wi, scores = torch.zeros((2, 4, 128), dtype=F16), torch.zeros((25, 128), dtype=F16), torch.ones((2, 4)), \
        torch.zeros((2, 28))
    return [
        ("pad_kv", 1, lambda **k: ds4a.pad_kv(r, 33, **k)),
        ("attn_prefill", 2, lambda **k: ds4a.attn_prefill(L, q, r, r, r, r, want_lse=True, **k)),
        ("attn_decode", 3, lambda **k: ds4a.attn_decode(L, q, r, r, r, r, want_lse=True, **k)),
        ("attn_decode_fp8", 2, lambda **k: ds4a.attn_decode_fp8(L, q, r, r, c, sc, c, sc, **k)),
        ("attn_decode_fp8kv", 2, lambda **k: ds4a.attn_decode_fp8kv(L, q, c, c, c, c, **f8, **k)),
        ("attn_prefill_fp8kv", 2, lambda **k: ds4a.attn_prefill_fp8kv(L, q, c, c, c, c, **f8, **k)),
        ("attn_decode_batch", 2, lambda **k: ds4a.attn_decode_batch(S, geom, q, b, b, b, b, **k)),
        ("attn_decode_partials", 1, lambda **k: ds4a.attn_decode_partials(L, q, r, r, r, r, **k)),
        ("attn_decode_noalloc", 1, lambda **k: ds4a.attn_decode_noalloc(L, q, r, r, r, r, **k)),
        ("attn_indexed", 1, lambda **k: ds4a.attn_indexed(L, q, r, r, r, r, idx, **k)),
        ("attn_indexed_fp8kv", 1, lambda **k: ds4a.attn_indexed_fp8kv(L, q, c, c, c, c, idx, **f8, **k)),
        ("indexer_scores", 1, lambda **k: ds4a.indexer_scores(L, qi, ki, wi, scale=1.0, **k)),
        ("indexer_topk", 1, lambda **k: ds4a.indexer_topk(L, scores, 8, **k)),
        ("compress_append", 1, lambda **k: ds4a.compress_append(kv, kv, state, state, 0, 4, **k)),
        ("quantize_kv_fp8", 2, lambda **k: ds4a.quantize_kv_fp8(r, **k)),
        ("attn_decode_paged", 3, lambda **k: ds4a.attn_decode_paged(SHAPE, geom, q, None, rows, want_lse=True, **k)),
        ("prepare_decode_paged", 1, lambda **k: ds4a.prepare_decode_paged(SHAPE, geom, q, None, rows, out=q, **k)),
        ("evict_paged", 3, lambda **k: ds4a.evict_paged(SHAPE, geom, rows, w, 10, **k)),
        ("rmsnorm_fp8", 4, lambda **k: ds4a.rmsnorm_fp8(x, one, residual=x, want_y=True, **k)),
    ]


@pytest.mark.parametrize("i", range(19))
def test_tensors_of_a_call_are_made_on_its_stream(monkeypatch, i):
    """A workspace freed to another stream's pool could be handed out while the call's kernels still use it."""
    name, n, call = wrapper_calls()[i]
    monkeypatch.setattr(ds4a, "_lib", Library())
    s = Streams(monkeypatch)
    for stream in (None, "side"):
        s.made.clear()
        call(stream=stream)
        assert [on for _, on in s.made] == [stream] * n and s.current is None, name
