"""What the operators around a paged key-value cache are measured on.

Five operators of one serving step over a paged cache (64 query heads, one shared K/V row of 512):

* ``decode``   one new token per sequence over its raw window rows and its compressed rows, both
               read through page tables (fp16 rows, or E4M3 codes with a scale per row);
* ``weights``  the attention weight each compressed row received in such a step, summed over the
               heads and added to what it received before;
* ``evict``    keeping the rows that received most, and moving kept rows into the freed slots;
* ``norm``     root-mean-square norm of (x + residual), as E4M3 codes with scales;
* ``append``   new K/V rows written into their cache slots (quantised where the cache is E4M3).

A case is a dict of plain values; ``run`` computes it in elementary torch operations, or, where
``own`` is true, with the calls a serving loop makes: built once on its buffers, then issued.
"""

import math

import numpy as np
import torch

own = False

H, D = 64, 512
WINDOW = 128
SCALE = 1.0 / math.sqrt(D)
E4M3_MAX = 448.0
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One sequence at 32K tokens of a ratio-128 layer: 256 compressed rows, the latency of a step.
        dict(name="decode_one_32k", op="decode", n_seq=1, rows=256, ratio=128, ragged=False, fp8=False, shared=False,
             page=64),
        # 64 requests of very different lengths in one step; K and V are the same row, as the engine stores it.
        dict(name="decode_64_ragged_shared", op="decode", n_seq=64, rows=2000, ratio=128, ragged=True, fp8=False,
             shared=True, page=16),
        # One very long context (a million tokens of a ratio-4 layer read in full).
        dict(name="decode_one_256k", op="decode", n_seq=1, rows=262144, ratio=4, ragged=False, fp8=False,
             shared=False, page=128),
        # 24 requests over an E4M3 cache, raw rows included.
        dict(name="decode_24_e4m3", op="decode", n_seq=24, rows=8192, ratio=4, ragged=True, fp8=True, shared=True,
             page=64),
        # The weights of one short sequence's step, and of a batch over E4M3 rows.
        dict(name="weights_one_2k", op="weights", n_seq=1, rows=2048, ratio=4, ragged=False, fp8=False, page=64),
        dict(name="weights_16_e4m3", op="weights", n_seq=16, rows=16384, ratio=4, ragged=True, fp8=True, page=64),
        # A cache held at its budget: every step frees one row of each of 64 sequences.
        dict(name="evict_step_64", op="evict", n_seq=64, rows=1025, keep=1024, ratio=128, ragged=False, fp8=True,
             page=64),
        # A long cache halved at once.
        dict(name="evict_half_2x128k", op="evict", n_seq=2, rows=131072, keep=65536, ratio=4, ragged=False, fp8=False,
             page=128),
        # The hidden stream of one token, and of a prefill chunk, with a scale per 128 values.
        dict(name="norm_1x4096", op="norm", n=1, width=4096, residual=True, group=128, f32=False),
        dict(name="norm_2048x4096", op="norm", n=2048, width=4096, residual=True, group=128, f32=False),
        # One step's K/V rows of 64 sequences into an E4M3 cache, and a prefill chunk's into an fp16 one.
        dict(name="append_64_e4m3", op="append", n=64, fp8=True, page=64, pages=256),
        dict(name="append_2048", op="append", n=2048, fp8=False, page=16, pages=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "weights", "evict", "norm", "append"])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    if op in ("decode", "weights"):
        n_seq = _log_int(rng, 1, 200)
        rows = _log_int(rng, 1, max(2, min(65536, 200000 // n_seq)))
        c = dict(op=op, n_seq=n_seq, rows=rows, ratio=rng.choice([1, 4, 128]), ragged=rng.random() < 0.7,
                 fp8=rng.random() < 0.5, page=page)
        if op == "decode":
            c["shared"] = rng.random() < 0.5
        return c
    if op == "evict":
        n_seq = _log_int(rng, 1, 128)
        rows = _log_int(rng, 2, max(4, min(131072, 200000 // n_seq)))
        return dict(op=op, n_seq=n_seq, rows=rows, keep=max(1, int(rows * rng.uniform(0.3, 1.0))), ratio=4,
                    ragged=rng.random() < 0.5, fp8=rng.random() < 0.5, page=page)
    if op == "norm":
        width = rng.choice([512, 1024, 1536, 4096, 7168, 8 * rng.randint(1, 1000)])
        return dict(op=op, n=_log_int(rng, 1, max(2, 8000000 // width)), width=width, residual=rng.random() < 0.6,
                    group=rng.choice([0, 64, 128]), f32=rng.random() < 0.4)
    n = _log_int(rng, 1, 4096)
    return dict(op=op, n=n, fp8=rng.random() < 0.5, page=page, pages=-(-2 * n // page) + rng.randint(0, 8))


def _lengths(case):
    """Compressed rows of each sequence: the case's rows, or a spread over a quarter of them and all."""
    n, rows = case["n_seq"], case["rows"]
    if not case["ragged"]:
        return [rows] * n
    return [max(1, int(rows * (0.25 + 0.75 * ((0.13 + 0.6180339887 * b) % 1.0)))) for b in range(n)]


def _positions(case):
    """The new token's position: its compressed rows have all ended, and a few positions have passed since."""
    return [c * case["ratio"] + min(case["ratio"] - 1, 1) + b % 7 for b, c in enumerate(_lengths(case))]


def _raw_rows(pos, page):
    """Raw rows kept: whole pages from the one where the window starts."""
    first = max(0, pos + 1 - WINDOW) // page * page
    return pos + 1 - first, first


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _codes(x):
    """E4M3 codes (uint8) and per-row scales of the last axis: scale = absmax / 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, E4M3_MAX / amax, torch.zeros_like(amax))
    q = (x * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), amax / E4M3_MAX


def _pool(g, n_pages, page, fp8):
    """Random rows [n_pages, page, 512] (rows differ in size as cache rows do), with their scales or None."""
    x = torch.empty((n_pages, page, D), dtype=torch.float16, device=DEV)
    for p in range(0, n_pages, 1024):
        y = torch.randn((min(1024, n_pages - p), page, D), generator=g, device=DEV)
        y *= 0.5 + torch.rand((y.shape[0], page, 1), generator=g, device=DEV)
        x[p:p + 1024] = y.half()
    if not fp8:
        return x, None
    codes = torch.empty((n_pages, page, D), dtype=torch.uint8, device=DEV)
    scale = torch.empty((n_pages, page), dtype=torch.float32, device=DEV)
    for p in range(0, n_pages, 1024):
        codes[p:p + 1024], scale[p:p + 1024] = _codes(x[p:p + 1024])
    return codes, scale


def _segment(g, counts, page, fp8, shared):
    """A pool with the pages of all sequences in random order, and the page tables."""
    per = [-(-c // page) for c in counts]
    width = max(max(per), 1)
    total = sum(per)
    order = torch.randperm(max(total, 1), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    first = np.concatenate([[0], np.cumsum(per)])
    at = torch.arange(width, device=DEV)[None, :] + torch.tensor(first[:-1], device=DEV)[:, None]
    have = torch.arange(width, device=DEV)[None, :] < torch.tensor(per, device=DEV)[:, None]
    table = torch.where(have, order[at.clamp(max=max(total, 1) - 1)], table).contiguous()
    k, ks = _pool(g, max(total, 1), page, fp8)
    v, vs = (k, ks) if shared else _pool(g, max(total, 1), page, fp8)
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, page=page)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("decode", "weights", "evict"):
        n = case["n_seq"]
        pos, comp = _positions(case), _lengths(case)
        raw = [_raw_rows(p, case["page"]) for p in pos]
        s["geom"] = torch.tensor([[p, r[0], r[1], c] for p, r, c in zip(pos, raw, comp)], dtype=torch.int32,
                                 device=DEV)
        s["comp"] = _segment(g, comp, case["page"], case["fp8"], op == "weights" or case.get("shared", False))
        cols = s["comp"]["table"].shape[1] * case["page"]
    if op in ("decode", "weights"):
        s["q"] = torch.randn((n, H, D), generator=g, device=DEV).half()
    if op == "decode":
        s["raw"] = _segment(g, [r[0] for r in raw], case["page"], case["fp8"], case["shared"])
        s["o"] = torch.zeros((n, H, D), dtype=torch.float16, device=DEV)
        s["lse"] = torch.zeros((n, H), dtype=torch.float32, device=DEV)
    elif op == "weights":
        spread = torch.tensor([math.log(c + WINDOW) + 0.7 for c in comp], device=DEV)
        s["lse"] = spread[:, None] + 0.2 * torch.randn((n, H), generator=g, device=DEV)
        s["acc"] = 4.0 * torch.rand((n, cols), generator=g, device=DEV)
        s["acc_out"] = torch.zeros((n, cols), dtype=torch.float32, device=DEV)
    elif op == "evict":
        # What rows received so far: a few receive most; many exactly nothing, so that ties are met.
        w = torch.randn((n, cols), generator=g, device=DEV).mul(2.0).exp()
        s["acc"] = torch.where(torch.rand((n, cols), generator=g, device=DEV) < 0.05, torch.zeros_like(w), w)
        s["ids"] = torch.arange(cols, dtype=torch.int32, device=DEV).expand(n, cols).contiguous()
        s["kept"] = torch.zeros((n, -(-case["keep"] // 4) * 4), dtype=torch.int32, device=DEV)[:, :case["keep"]]
        s["acc_out"] = torch.zeros((n, cols), dtype=torch.float32, device=DEV)
        s["ids_out"] = torch.zeros((n, cols), dtype=torch.int32, device=DEV)
        s["n_out"] = torch.zeros((n,), dtype=torch.int32, device=DEV)
    elif op == "norm":
        n, width = case["n"], case["width"]
        dt = torch.float32 if case["f32"] else torch.float16
        s["x"] = torch.randn((n, width), generator=g, device=DEV).to(dt)
        s["w"] = 1.0 + 0.2 * torch.randn((width,), generator=g, device=DEV)
        s["res"] = (3.0 * torch.randn((n, width), generator=g, device=DEV)).to(dt) if case["residual"] else None
        groups = 1 if case["group"] == 0 else -(-width // case["group"])
        s["res_out"] = torch.zeros((n, width), dtype=dt, device=DEV) if case["residual"] else None
        s["codes"] = torch.zeros((n, -(-width // 16) * 16), dtype=torch.uint8, device=DEV)[:, :width]
        s["scales"] = torch.zeros((n, groups), dtype=torch.float32, device=DEV)
    else:
        n, page, pages = case["n"], case["page"], case["pages"]
        s["k_new"] = torch.randn((n, D), generator=g, device=DEV).half()
        s["v_new"] = torch.randn((n, D), generator=g, device=DEV).half()
        s["slots"] = torch.randperm(page * pages, generator=g, device=DEV)[:n].to(torch.int32)
        s["slots"] = torch.where(torch.arange(n, device=DEV) % 16 == 15, -1, s["slots"]).to(torch.int32)  # padding
        k, ks = _pool(g, pages, page, case["fp8"])
        v, vs = _pool(g, pages, page, case["fp8"])
        s["pool"] = dict(k=k, v=v, ks=ks, vs=vs, table=None, page=page)
    if own:
        s["step"] = _own_step(s)  # the arguments of the loop's call on these buffers
    return s


# ------------------------------------------------------------------ the framework's calls

def _own_step(s):
    from mqa_flash_attention_gb300 import ds4a
    case, op = s["case"], s["case"]["op"]

    def rows(p):
        return ds4a.PagedRows(p["k"], p["v"], p["table"], k_scale=p["ks"], v_scale=p["vs"])

    if op in ("decode", "weights", "evict"):
        shape = dict(T=1, q_pos0=0, n_raw=0, raw_pos0=0, n_comp=0, ratio=case["ratio"], window=WINDOW, scale=SCALE)
    if op == "decode":
        raw, comp = rows(s["raw"]), rows(s["comp"])
        ws = torch.empty(ds4a.decode_paged_workspace_bytes(case["n_seq"], shape, raw, comp), dtype=torch.uint8,
                         device=DEV)
        return ds4a.prepare_decode_paged(shape, s["geom"], s["q"], raw, comp, workspace=ws, out=s["o"], lse=s["lse"])
    if op == "weights":
        return ds4a.prepare_weights_paged(shape, s["geom"], s["q"], rows(s["comp"]), s["lse"], weights=s["acc"],
                                          decay=0.98, out=s["acc_out"])
    if op == "evict":
        ws = torch.empty(ds4a.evict_paged_workspace_bytes(case["n_seq"], case["keep"]), dtype=torch.uint8, device=DEV)
        return ds4a.prepare_evict_paged(shape, s["geom"], rows(s["comp"]), s["acc"], case["keep"],
                                        n_recent=min(32, case["keep"] // 4), n_first=min(4, case["keep"] // 4),
                                        ids=s["ids"], kept=s["kept"], weights_out=s["acc_out"], ids_out=s["ids_out"],
                                        n_out=s["n_out"], workspace=ws)
    if op == "norm":
        return ds4a.prepare_rmsnorm_fp8(s["x"], s["w"], eps=1e-6, residual=s["res"], residual_out=s["res_out"],
                                        group=case["group"], codes=s["codes"], scales=s["scales"])
    return ds4a.prepare_append_paged(rows(s["pool"]), s["k_new"], s["v_new"], s["slots"])


# ------------------------------------------------------------------ plain forms

def _values(pool, scale):
    """Row values of a pool in 32 bits."""
    if scale is None:
        return pool.float()
    return pool.view(torch.float8_e4m3fn).float() * scale[..., None]


def _gather(seg, n, which):
    """Rows 0 .. n-1 of every sequence through its page table: [n_seq, n, 512] in 32 bits."""
    j = torch.arange(n, device=DEV)
    page = seg["table"][:, j // seg["page"]].long().clamp(min=0)
    slot = (j % seg["page"])[None, :]
    rows = seg[which][page, slot]
    scale = seg[which + "s"]
    return _values(rows, None if scale is None else scale[page, slot])


def _seen(s):
    """Which raw and compressed rows each sequence's token sees."""
    g, case = s["geom"].long(), s["case"]
    pos, n_raw, raw0, n_comp = g[:, 0:1], g[:, 1:2], g[:, 2:3], g[:, 3:4]
    nr = s["raw"]["table"].shape[1] * case["page"] if "raw" in s else 0
    nc = s["comp"]["table"].shape[1] * case["page"]
    i, c = torch.arange(nr, device=DEV)[None, :], torch.arange(nc, device=DEV)[None, :]
    raw = (i < n_raw) & (raw0 + i <= pos) & (raw0 + i > pos - WINDOW)
    comp = (c < n_comp) & ((c + 1) * case["ratio"] <= pos + 1)
    return raw, comp


def _decode(s):
    raw, comp = _seen(s)
    q = s["q"].float()
    seen = torch.cat([raw, comp], 1)[:, None, :]
    k = torch.cat([_gather(s["raw"], raw.shape[1], "k"), _gather(s["comp"], comp.shape[1], "k")], 1)
    x = (q @ k.transpose(1, 2)) * SCALE
    del k
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.cat([_gather(s["raw"], raw.shape[1], "v"), _gather(s["comp"], comp.shape[1], "v")], 1)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return {"o": o.half(), "lse": (top + total.log())[..., 0]}


def _weights(s):
    _, comp = _seen(s)
    k = _gather(s["comp"], comp.shape[1], "k")
    x = (s["q"].float() @ k.transpose(1, 2)) * SCALE
    w = (x - s["lse"][:, :, None]).exp().sum(1)
    return {"acc": torch.where(comp, 0.98 * s["acc"] + w, s["acc_out"])}


def _order(s):
    """Rank keys: a protected row above every other, absent rows below; larger is kept first."""
    case, g = s["case"], s["geom"].long()
    w = torch.where(torch.isnan(s["acc"]), torch.full_like(s["acc"], -math.inf), s["acc"]) + 0.0
    bits = w.view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    n_recent, n_first = min(32, case["keep"] // 4), min(4, case["keep"] // 4)
    ended = (g[:, 0:1] + 1) // case["ratio"]
    safe = (s["ids"] < n_first) | (s["ids"] >= ended - n_recent)
    key = torch.where(safe, torch.full_like(key, 1 << 33), key)
    j = torch.arange(key.shape[1], device=DEV)[None, :]
    return torch.where(j < g[:, 3:4], key, torch.full_like(key, -(1 << 33)))


def _evict(s):
    case, seg = s["case"], s["comp"]
    keep, n = case["keep"], s["geom"][:, 3:4].long()
    key = _order(s)
    cols = key.shape[1]
    take = min(keep, cols)
    n_out = n.clamp(max=keep)
    best = key.sort(dim=1, descending=True, stable=True).indices[:, :take]
    among = torch.arange(take, device=DEV)[None, :] < n_out
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(1, best, among)
    j = torch.arange(cols, device=DEV)[None, :].expand_as(key)
    moves, hole = kept & (j >= n_out), ~kept & (j < n_out)
    # The h-th freed slot below n_out takes the h-th kept row from above it.
    to = torch.where(moves, moves.long().cumsum(1) - 1, torch.full_like(key, cols))
    mover = torch.zeros((key.shape[0], cols + 1), dtype=torch.long, device=DEV).scatter_(1, to, j)
    src = torch.where(hole, mover.gather(1, (hole.long().cumsum(1) - 1).clamp(min=0)), j)
    live = j < n_out
    b, i = hole.nonzero(as_tuple=True)
    f, p = src[b, i], seg["page"]
    dst_at = (seg["table"][b, i // p].long(), i % p)
    src_at = (seg["table"][b, f // p].long(), f % p)
    for name in ("k", "v", "ks", "vs"):
        if seg[name] is not None:
            seg[name][dst_at] = seg[name][src_at]
    acc = torch.where(live, s["acc"].gather(1, src), s["acc_out"])
    ids = torch.where(live, s["ids"].gather(1, src.clamp(max=cols - 1)), s["ids_out"])
    pad = torch.full((key.shape[0], keep - take), -1, dtype=torch.int32, device=DEV)
    listed_rows = torch.cat([torch.where(live, src, torch.full_like(src, -1))[:, :take].to(torch.int32), pad], 1)
    return _evict_out(s, listed_rows, acc, ids, n_out[:, 0].to(torch.int32))


def _evict_out(s, kept, acc, ids, n_out):
    seg = s["comp"]
    out = {"kept": kept, "acc": acc, "ids": ids, "n": n_out}
    for name in ("k", "v"):
        out[name] = seg[name] if seg[name + "s"] is None else seg[name].view(torch.float8_e4m3fn)
        if seg[name + "s"] is not None:
            out[name + "_scale"] = seg[name + "s"]
    return out


def _norm(s):
    case = s["case"]
    h = s["x"].float()
    out = {}
    if s["res"] is not None:
        h = h + s["res"].float()
        out["residual"] = h.to(s["x"].dtype)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w"]
    n, width = y.shape
    group = width if case["group"] == 0 else case["group"]
    groups = -(-width // group)
    z = torch.zeros((n, groups * group), device=DEV)
    z[:, :width] = y
    codes, scale = _codes(z.view(n, groups, group))
    out["codes"] = codes.view(n, groups * group)[:, :width].contiguous().view(torch.float8_e4m3fn)
    out["scales"] = scale
    return out


def _append(s):
    pool, at = s["pool"], s["slots"].long()
    have = (at >= 0).nonzero()[:, 0]
    at = at[have]
    where = (at // pool["page"], at % pool["page"])
    for name in ("k", "v"):
        new = s[name + "_new"][have]
        if pool[name + "s"] is None:
            pool[name][where] = new
        else:
            pool[name][where], pool[name + "s"][where] = _codes(new)
    return _append_out(s)


def _append_out(s):
    pool = s["pool"]
    if pool["ks"] is None:
        return {"k": pool["k"], "v": pool["v"]}
    f8 = torch.float8_e4m3fn
    return {"k": pool["k"].view(f8), "v": pool["v"].view(f8), "k_scale": pool["ks"], "v_scale": pool["vs"]}


_PLAIN = {"decode": _decode, "weights": _weights, "evict": _evict, "norm": _norm, "append": _append}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    s["step"]()
    if op == "decode":
        return {"o": s["o"], "lse": s["lse"]}
    if op == "weights":
        return {"acc": s["acc_out"]}
    if op == "evict":
        return _evict_out(s, s["kept"], s["acc_out"], s["ids_out"], s["n_out"])
    if op == "norm":
        out = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
        return out if s["res"] is None else dict(out, residual=s["res_out"])
    return _append_out(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("decode", "weights"):
        n, row = case["n_seq"], (D + 4 if case["fp8"] else 2 * D)
        comp = sum(_lengths(case))
        if op == "weights":
            return {"bytes": comp * (row + 8) + n * H * (2 * D + 4), "flops": 2 * H * D * comp}
        rows = comp + sum(min(WINDOW, p + 1) for p in _positions(case))
        return {"bytes": rows * row * (1 if case["shared"] else 2) + n * H * (4 * D + 4), "flops": 4 * H * D * rows}
    if op == "evict":
        n, row = case["n_seq"], (D + 4 if case["fp8"] else 2 * D)
        total = sum(_lengths(case))
        out = sum(min(c, case["keep"]) for c in _lengths(case))
        # A kept row above the budget moves: a row is kept with the share that the budget leaves.
        moved = sum(max(0, c - case["keep"]) * min(1.0, case["keep"] / c) for c in _lengths(case))
        return {"bytes": total * 8 + out * 12 + moved * 4 * row, "flops": total}
    if op == "norm":
        n, width, size = case["n"], case["width"], 4 if case["f32"] else 2
        groups = 1 if case["group"] == 0 else -(-width // case["group"])
        return {"bytes": n * (width * (size * (3 if case["residual"] else 1) + 1) + 4 * groups) + 4 * width,
                "flops": 6 * n * width}
    n = case["n"] - case["n"] // 16  # every sixteenth row is padding
    return {"bytes": 2 * n * (2 * D + (D + 4 if case["fp8"] else 2 * D)) + 4 * case["n"], "flops": 4 * n * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_codes(y):
    """The E4M3 numbers nearest to y * 448 / absmax over the last axis (ties to even), and the scales."""
    amax = y.abs().amax(-1, keepdim=True)
    x = y * (E4M3_MAX / amax.clamp(min=1e-300))
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (x / step).round() * step, amax[..., 0] / E4M3_MAX


def _exact_rows(seg, b, n, which):
    """Rows 0 .. n-1 of sequence b, page by page."""
    if n == 0:
        return torch.zeros((0, D), dtype=torch.float64, device=DEV)
    pages = seg["table"][b, : -(-n // seg["page"])].long()
    rows = seg[which][pages].reshape(-1, D)[:n]
    if seg[which + "s"] is None:
        return rows.double()
    return rows.view(torch.float8_e4m3fn).double() * seg[which + "s"][pages].reshape(-1)[:n, None].double()


def exact(case, seed):
    global own
    kept_own, own = own, False
    s = prepare(case, seed)
    own = kept_own
    op = case["op"]
    if op == "evict":
        return None  # whole numbers and moved rows: nothing is rounded
    if op == "append":
        if not case["fp8"]:
            return None
        out = {}
        for name in ("k", "v"):
            vals = s["pool"][name].view(torch.float8_e4m3fn).double().reshape(-1, D)
            scale = s["pool"][name + "s"].double().reshape(-1)
            at = s["slots"].long()
            new, sc = _exact_codes(s[name + "_new"].double())
            vals[at[at >= 0]], scale[at[at >= 0]] = new[at >= 0], sc[at >= 0]
            out[name], out[name + "_scale"] = vals.view(s["pool"][name].shape), scale.view(s["pool"][name].shape[:2])
        return out
    if op == "norm":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + 1e-6) * s["w"].double()
        width = y.shape[1]
        group = case["group"] or width
        parts = [_exact_codes(y[:, c:c + group]) for c in range(0, width, group)]
        out = {"codes": torch.cat([p[0] for p in parts], 1), "scales": torch.stack([p[1] for p in parts], 1)}
        return out if s["res"] is None else dict(out, residual=h)
    o, lse, acc = [], [], s["acc_out"].double() if op == "weights" else None
    geom = s["geom"].tolist()
    for b, (pos, n_raw, raw0, n_comp) in enumerate(geom):
        n_comp = min(n_comp, (pos + 1) // case["ratio"])
        q = s["q"][b].double()
        if op == "weights":
            k = _exact_rows(s["comp"], b, n_comp, "k")
            p = torch.exp(q @ k.T / math.sqrt(D) - s["lse"][b].double()[:, None])
            acc[b, :n_comp] = s["acc"][b, :n_comp].double() * 0.98 + p.sum(0)
            continue
        lo, hi = max(0, pos + 1 - WINDOW - raw0), min(n_raw, pos + 1 - raw0)
        k = torch.cat([_exact_rows(s["raw"], b, n_raw, "k")[lo:hi], _exact_rows(s["comp"], b, n_comp, "k")])
        v = torch.cat([_exact_rows(s["raw"], b, n_raw, "v")[lo:hi], _exact_rows(s["comp"], b, n_comp, "v")])
        x = q @ k.T / math.sqrt(D)
        lse.append(torch.logsumexp(x, 1))
        o.append(torch.softmax(x, 1) @ v)
    return {"acc": acc} if op == "weights" else {"o": torch.stack(o), "lse": torch.stack(lse)}
