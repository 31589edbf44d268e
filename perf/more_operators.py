"""What the operators of a step with several new tokens per sequence are measured on.

Four operators around a paged key-value cache (64 query heads, one shared K/V row of 512), in the order in
which a serving step with drafted tokens, or with prompts of different lengths, makes them:

* ``pages``   page tables and slots from the rows each sequence has and wants: pages taken from a free list,
              pages given back (a window's leading pages among them), the slots of the new rows;
* ``tree``    attention of the new tokens, packed over the sequences: a tree of drafted tokens per sequence, each
              seeing its ancestors, or (without parents) a run of a prompt, causal; over raw window rows and
              compressed rows, both through page tables (fp16, or E4M3 codes with a scale per row);
* ``accept``  the path of drafted tokens that agree with what the model chose;
* ``commit``  the accepted tokens' K/V rows moved to the places behind the cached ones.

A case is a dict of plain values; ``run`` computes it in elementary torch operations, or, where ``own`` is true,
with the calls a serving loop makes: built once on its buffers, then issued.
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
        # Eight drafted tokens of one request at 32K positions of a ratio-128 layer: the latency of a step.
        dict(name="tree_1x8_32k", op="tree", n_seq=1, new=8, rows=256, ratio=128, chain=False, ragged=False, fp8=False,
             shared=True, page=64),
        # 32 requests of different lengths, up to 16 drafted tokens each, K and V the same row.
        dict(name="tree_32x16_ragged", op="tree", n_seq=32, new=16, rows=4000, ratio=4, chain=False, ragged=True,
             fp8=False, shared=True, page=64),
        # Wide trees over an E4M3 cache.
        dict(name="tree_8x64_e4m3", op="tree", n_seq=8, new=64, rows=8192, ratio=4, chain=False, ragged=True, fp8=True,
             shared=True, page=64),
        # One very long context, K and V apart (half a million tokens of a ratio-4 layer read in full).
        dict(name="tree_1x16_128k", op="tree", n_seq=1, new=16, rows=131072, ratio=4, chain=False, ragged=False,
             fp8=False, shared=False, page=128),
        # Runs of seven prompts of different lengths in one call, on a ratio-128 layer.
        dict(name="prompt_7_ragged_r128", op="tree", n_seq=7, new=700, rows=300, ratio=128, chain=True, ragged=True,
             fp8=False, shared=True, page=16),
        # A 2048-token run of one prompt at position 30720, every compressed row of a ratio-4 layer read.
        dict(name="prompt_2048_r4", op="tree", n_seq=1, new=2048, rows=7680, ratio=4, chain=True, ragged=False, fp8=False,
             shared=True, page=64),
        # Room for eight drafted rows of 64 requests, then given back; and a large batch of prompts admitted at
        # once, its windows' leading pages dropped.
        dict(name="pages_64_drafts", op="pages", n_seq=64, rows=4000, new=8, page=64, drop=False, spare=2.0),
        dict(name="pages_1024_prompts", op="pages", n_seq=1024, rows=300, new=500, page=16, drop=True, spare=2.0),
        # Acceptance of one request's drafts, and of a large batch with wide trees.
        dict(name="accept_1x8", op="accept", n_seq=1, new=8, chain=False),
        dict(name="accept_512x64", op="accept", n_seq=512, new=64, chain=False),
        # Accepted rows of 32 requests (fp16, K and V apart), and of 256 in an E4M3 cache.
        dict(name="commit_32x16", op="commit", n_seq=32, new=16, fp8=False, shared=False, page=64),
        dict(name="commit_256x64_e4m3", op="commit", n_seq=256, new=64, fp8=True, shared=False, page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tree", "pages", "accept", "commit"])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128])
    if op == "tree":
        chain = rng.random() < 0.4
        n_seq = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(2, (2048 if chain else 1024) // n_seq)) if chain or n_seq > 8 else _log_int(rng, 1, 128)
        rows = _log_int(rng, 1, max(2, min(131072 // n_seq, 6000000 // (n_seq * new))))
        return dict(op=op, n_seq=n_seq, new=new, rows=rows, ratio=rng.choice([1, 4, 128]), chain=chain,
                    ragged=rng.random() < 0.7, fp8=rng.random() < 0.4, shared=rng.random() < 0.6, page=page)
    if op == "pages":
        n_seq = _log_int(rng, 1, 1024)
        return dict(op=op, n_seq=n_seq, rows=_log_int(rng, 1, max(2, min(8000, 400000 // n_seq))),
                    new=_log_int(rng, 1, max(2, min(2000, 400000 // n_seq))), page=page, drop=rng.random() < 0.5,
                    spare=rng.choice([0.5, 1.0, 2.0]))
    n_seq, new = _log_int(rng, 1, 512), _log_int(rng, 1, 64)
    if op == "accept":
        return dict(op=op, n_seq=n_seq, new=new, chain=rng.random() < 0.3)
    return dict(op=op, n_seq=min(n_seq, 256), new=new, fp8=rng.random() < 0.5, shared=rng.random() < 0.5, page=page)


def _spread(b):
    return (0.13 + 0.6180339887 * b) % 1.0


def _new(case):
    """New tokens of each sequence: the case's, or a spread over a fifth of them and all."""
    n, new = case["n_seq"], case["new"]
    if not case.get("ragged", n > 1):
        return [new] * n
    return [max(1, int(round(new * (0.2 + 0.8 * _spread(b + 5))))) for b in range(n)]


def _lengths(case):
    """Compressed rows of each sequence before the new tokens."""
    n, rows = case["n_seq"], case["rows"]
    if not case["ragged"]:
        return [rows] * n
    return [max(1, int(rows * (0.25 + 0.75 * _spread(b)))) for b in range(n)]


def _geometry(case):
    """Per sequence (position of the first new token, cached raw rows, position of raw row 0, compressed rows).
    A prompt's run has the compressed rows of its own tokens too; those of drafts come with their acceptance."""
    out = []
    for b, (c, n) in enumerate(zip(_lengths(case), _new(case))):
        pos = c * case["ratio"] + min(case["ratio"] - 1, b % 3)
        first = max(0, pos + 1 - WINDOW) // case["page"] * case["page"]
        out.append((pos, pos - first, first, (pos + n) // case["ratio"] if case["chain"] else c))
    return out


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _trees(r, counts, chain):
    """Parents of the packed nodes, counted within their sequence; -1: a root."""
    out = []
    for n in counts:
        t = np.arange(n)
        if chain:
            out.append(t - 1)
            continue
        back = 1 + (r.random(n) * np.minimum(t, 8)).astype(np.int64)
        p = np.where(r.random(n) < 0.04, -1, t - back)
        p[0] = -1
        out.append(np.maximum(p, -1))
    return np.concatenate(out).astype(np.int32)


def _first(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


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


def _table(g, per, width):
    """Tables of per[b] pages each, all different, in random order; -1 behind them."""
    order = torch.randperm(max(sum(per), 1), generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.concatenate([[0], np.cumsum(per)])[:-1], device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    have = at < torch.tensor(per, device=DEV)[:, None]
    return torch.where(have, order[(at + first[:, None]).clamp(max=max(sum(per), 1) - 1)], -1).to(torch.int32).contiguous()


def _segment(g, counts, page, fp8, shared):
    """A pool with the pages of all sequences in random order, and the page tables."""
    per = [-(-c // page) for c in counts]
    table = _table(g, per, max(max(per), 1))
    k, ks = _pool(g, max(sum(per), 1), page, fp8)
    v, vs = (k, ks) if shared else _pool(g, max(sum(per), 1), page, fp8)
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, page=page)


def prepare(case, seed):
    g, r = _gen(seed), np.random.RandomState((int(seed) * 7919 + 11) % (1 << 31))
    s = dict(case=case)
    op = case["op"]
    if op == "pages":
        _prepare_pages(s, case, g)
    else:
        new = _new(case)
        s["first"] = _first(new)
        s["new"] = new
    if op == "tree":
        geom = _geometry(case)
        s["parent"] = None if case["chain"] else torch.tensor(_trees(r, new, False), device=DEV)
        s["geom"] = torch.tensor(geom, dtype=torch.int32, device=DEV)
        s["comp"] = _segment(g, [x[3] for x in geom], case["page"], case["fp8"], case["shared"])
        s["raw"] = _segment(g, [x[1] + n for x, n in zip(geom, new)], case["page"], case["fp8"], case["shared"])
        s["q"] = torch.randn((sum(new), H, D), generator=g, device=DEV).half()
        s["o"] = torch.zeros((sum(new), H, D), dtype=torch.float16, device=DEV)
        s["lse"] = torch.zeros((sum(new), H), dtype=torch.float32, device=DEV)
    elif op == "accept":
        _prepare_accept(s, case, r)
    elif op == "commit":
        # Each sequence accepts a path through its tree: rows behind the cached ones of its window.
        n_raw = [WINDOW + b % case["page"] for b in range(case["n_seq"])]
        s["geom"] = torch.tensor([[n, n, 0, 0] for n in n_raw], dtype=torch.int32, device=DEV)
        path = np.full((case["n_seq"], case["new"]), -1, dtype=np.int32)
        count = np.zeros(case["n_seq"], dtype=np.int32)
        for b, n in enumerate(new):
            took = np.flatnonzero(r.random(n) < 0.35)
            path[b, :len(took)], count[b] = took, len(took)
        s["path"], s["count"] = torch.tensor(path, device=DEV), torch.tensor(count, device=DEV)
        s["pool"] = _segment(g, [a + n for a, n in zip(n_raw, new)], case["page"], case["fp8"], case["shared"])
    if own:
        s["step"] = _own_step(s)  # the calls of the loop on these buffers
    return s


def _prepare_pages(s, case, g):
    n, page = case["n_seq"], case["page"]
    u, v = (np.array([_spread(k * b + k) for b in range(n)]) for k in (1, 2))
    have = np.maximum(1, (case["rows"] * (0.25 + 0.75 * u)).astype(np.int64))
    grow = (case["new"] * (0.2 + 0.8 * v)).astype(np.int64)
    b = np.arange(n)
    want = np.where(b % 10 == 7, have // 2, have + np.where(b % 10 == 3, 0, grow))  # some finish, or are cut back
    drop = np.where(b % 2 == 1, have // 3, 0) if case["drop"] else np.zeros(n, dtype=np.int64)
    held = -(-have // page)
    width = int(max(-(-np.maximum(have, want) // page)))
    spare = max(1, int(case["spare"] * (-(-want // page) - held).clip(min=0).sum()))
    n_pages = int(held.sum()) + spare
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["n_pages"] = n_pages
    first = torch.tensor(np.concatenate([[0], np.cumsum(held)])[:-1], device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    own_pages = at < torch.tensor(held, device=DEV)[:, None]
    s["table"] = torch.where(own_pages, order[(at + first[:, None]).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    s["free"] = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    s["free"][:spare] = order[n_pages - spare:]
    s["n_free"] = torch.tensor([spare], dtype=torch.int32, device=DEV)
    gone = np.minimum(drop, have) // page * page
    after = np.maximum(want, gone) - gone  # rows after the first call, which gives the tables' new numbering
    for name, x in (("have", have), ("want", want), ("drop", drop), ("after", after)):
        s[name] = torch.tensor(x, dtype=torch.int32, device=DEV)
    rows = int((want - have).clip(min=0).sum())
    back = int((have - after).clip(min=0).sum())
    for name, m in (("1", rows), ("2", back)):
        s["slots" + name] = torch.zeros((m + 7,), dtype=torch.int32, device=DEV)  # a padded batch
        s["first" + name] = torch.zeros((n + 1,), dtype=torch.int32, device=DEV)
        s["short" + name] = torch.zeros((1,), dtype=torch.int32, device=DEV)


def _prepare_accept(s, case, r):
    """Drafted tokens that the model mostly agrees with: after most nodes it chose what one of the children holds."""
    counts = s["new"]
    parent = _trees(r, counts, case["chain"])
    n = len(parent)
    base = np.repeat(np.concatenate([[0], np.cumsum(counts)])[:-1], counts)
    token = r.randint(0, 100000, n)
    target = r.randint(0, 100000, n)
    up = np.where(parent >= 0, parent + base, -1)
    agree = r.random(n) < 0.75
    for t in r.permutation(n):  # a later write wins: the choice falls on any of the children
        if up[t] >= 0 and agree[up[t]]:
            target[up[t]] = token[t]
    prev = r.randint(0, 100000, case["n_seq"])
    heads = np.concatenate([[0], np.cumsum(counts)])[:-1]
    prev = np.where(r.random(case["n_seq"]) < 0.9, token[heads], prev)
    i32 = dict(dtype=torch.int32, device=DEV)
    s["parent"] = None if case["chain"] else torch.tensor(parent, **i32)
    for name, x in (("token", token), ("target", target), ("prev", prev)):
        s[name] = torch.tensor(x, **i32)
    s["path"] = torch.zeros((case["n_seq"], max(counts)), **i32)
    s["count"] = torch.zeros((case["n_seq"],), **i32)
    s["next"] = torch.zeros((case["n_seq"],), **i32)


# ------------------------------------------------------------------ the framework's calls

def _own_step(s):
    from mqa_flash_attention_gb300 import ds4a
    case, op = s["case"], s["case"]["op"]

    def rows(p):
        return ds4a.PagedRows(p["k"], p["v"], p["table"], k_scale=p["ks"], v_scale=p["vs"])

    if op == "tree":
        shape = dict(T=1, q_pos0=0, n_raw=0, raw_pos0=0, n_comp=0, ratio=case["ratio"], window=WINDOW, scale=SCALE)
        ws = torch.empty(ds4a.tree_paged_workspace_bytes(case["n_seq"], s["q"].shape[0]), dtype=torch.uint8, device=DEV)
        return ds4a.prepare_tree_paged(shape, s["geom"], s["first"], s["q"], rows(s["raw"]), rows(s["comp"]),
                                       parent=s["parent"], workspace=ws, out=s["o"], lse=s["lse"])
    if op == "pages":
        ws = torch.empty(ds4a.page_tables_workspace_bytes(case["n_seq"]), dtype=torch.uint8, device=DEV)
        one = ds4a.prepare_page_tables(s["table"], s["free"], s["n_free"], s["have"], s["want"], case["page"],
                                       drop=s["drop"] if case["drop"] else None, slots=s["slots1"], first=s["first1"],
                                       n_short=s["short1"], workspace=ws)
        two = ds4a.prepare_page_tables(s["table"], s["free"], s["n_free"], s["after"], s["have"], case["page"],
                                       slots=s["slots2"], first=s["first2"], n_short=s["short2"], workspace=ws)

        def step():
            one()
            two()
        return step
    if op == "accept":
        return ds4a.prepare_tree_accept(s["first"], s["token"], s["target"], parent=s["parent"], prev=s["prev"],
                                        path=s["path"], n_accepted=s["count"], next_token=s["next"])
    return ds4a.prepare_commit_paged(rows(s["pool"]), s["geom"], s["path"], s["count"])


# ------------------------------------------------------------------ plain forms

def _values(pool, scale):
    """Row values of a pool in 32 bits."""
    if scale is None:
        return pool.float()
    return pool.view(torch.float8_e4m3fn).float() * scale[..., None]


def _gather(seg, b, n, which):
    """Rows 0 .. n-1 of sequence b through its page table: [n, 512] in 32 bits."""
    j = torch.arange(n, device=DEV)
    page, slot = seg["table"][b, j // seg["page"]].long(), j % seg["page"]
    scale = seg[which + "s"]
    return _values(seg[which][page, slot], None if scale is None else scale[page, slot])


def _depths(parent, n):
    """Depth of each node, and which nodes are its ancestors or itself: [n, n]."""
    t = torch.arange(n, device=DEV)
    if parent is None:
        return t, t[None, :] <= t[:, None]
    seen = torch.eye(n, dtype=torch.bool, device=DEV)
    at = parent.long()
    for _ in range(n):  # one generation up at a time, all nodes together
        seen |= (at[:, None] == t[None, :])
        at = torch.where(at >= 0, parent.long()[at.clamp(min=0)], at)
    return seen.sum(1) - 1, seen


def _tree(s):
    case, first = s["case"], 0
    o, lse = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
    for b, ((pos, n_raw, raw0, n_comp), n) in enumerate(zip(_geometry(case), s["new"])):
        depth, anc = _depths(None if s["parent"] is None else s["parent"][first:first + n], n)
        p = pos + depth
        held = raw0 + torch.arange(n_raw, device=DEV)
        c = torch.arange(n_comp, device=DEV)
        seen = torch.cat([(held[None] <= p[:, None]) & (held[None] > p[:, None] - WINDOW),
                          anc & (depth[None] > depth[:, None] - WINDOW),
                          (c[None] + 1) * case["ratio"] <= p[:, None] + 1], 1)
        k = torch.cat([_gather(s["raw"], b, n_raw + n, "k"), _gather(s["comp"], b, n_comp, "k")])
        v = torch.cat([_gather(s["raw"], b, n_raw + n, "v"), _gather(s["comp"], b, n_comp, "v")])
        step = max(1, (1 << 28) // (H * len(k)))
        for t in range(0, n, step):
            q = s["q"][first + t:first + min(n, t + step)].float()
            x = (q.reshape(-1, D) @ k.T).view(len(q), H, -1) * SCALE
            x = x.masked_fill(~seen[t:t + step, None, :], -math.inf)
            top = x.amax(-1, keepdim=True)
            w = (x - top).exp()
            total = w.sum(-1, keepdim=True)
            y = (w.reshape(-1, w.shape[-1]) @ v).view(len(q), H, D) / total
            o[first + t:first + t + len(q)] = y.half()
            lse[first + t:first + t + len(q)] = (top + total.log())[..., 0]
        first += n
    return {"o": o, "lse": lse}


def _resize(s, have, want, drop, slots):
    """One call on the tables and the free list: new tables, list and count, then slots, first and what was short."""
    page, n_pages = s["case"]["page"], s["n_pages"]
    table, free = s["table"], s["free"]
    n, width = table.shape
    h, w = have.long(), want.long()
    gone = torch.minimum(drop.long(), h) // page
    held, need = (h + page - 1) // page, torch.maximum((w + page - 1) // page, gone)
    at = torch.arange(width, device=DEV)[None, :]
    back = ((at < gone[:, None]) | (at >= need[:, None]) & (at < held[:, None])) & (table >= 0) & (table < n_pages)
    given = table[back]
    top = int(s["n_free"]) + given.numel()
    free = free.clone()
    free[top - given.numel():top] = given
    after = torch.where(at < held[:, None], table, -1)
    new = (at >= held[:, None]) & (at < need[:, None])
    b, i = new.nonzero(as_tuple=True)
    k = top - 1 - torch.arange(len(b), device=DEV)
    after[b, i] = torch.where(k >= 0, free[k.clamp(min=0)], -1)
    grown = (w - h).clamp(min=0)
    first = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), grown.cumsum(0)])
    total = int(first[-1])
    owner = torch.repeat_interleave(torch.arange(n, device=DEV), grown)
    row = h[owner] + torch.arange(total, device=DEV) - first[owner]
    pg = after[owner, row // page]
    out = torch.full((slots.numel(),), -1, dtype=torch.int32, device=DEV)
    out[:total] = torch.where(pg >= 0, pg * page + row % page, -1).to(torch.int32)
    src = (at + gone[:, None]).clamp(max=width - 1)
    moved = torch.where(at < (need - gone)[:, None], after.gather(1, src), -1)
    used = torch.maximum(held, need - gone)
    s["table"].copy_(torch.where(at < used[:, None], moved, table))
    s["free"].copy_(free)
    s["n_free"].fill_(max(0, top - len(b)))
    return out, first.to(torch.int32), torch.tensor([max(0, len(b) - top)], dtype=torch.int32, device=DEV)


def _pages(s):
    out = {}
    none = torch.zeros_like(s["have"])
    out["slots1"], out["first1"], out["short1"] = _resize(s, s["have"], s["want"], s["drop"], s["slots1"])
    out["slots2"], out["first2"], out["short2"] = _resize(s, s["after"], s["have"], none, s["slots2"])
    return _pages_out(s, out)


def _pages_out(s, x):
    return {"table": s["table"], "free": s["free"], "n_free": s["n_free"],
            **{n + k: x[n + k] for n in ("slots", "first", "short") for k in "12"}}


def _accept(s):
    counts = torch.tensor(s["new"], device=DEV)
    n, width = len(s["new"]), s["path"].shape[1]
    nodes = int(counts.sum())
    owner = torch.repeat_interleave(torch.arange(n, device=DEV), counts)
    local = torch.arange(nodes, device=DEV) - s["first"].long()[owner]
    parent = local - 1 if s["parent"] is None else s["parent"].long()
    at = torch.full((n,), -1, dtype=torch.long, device=DEV)       # the last accepted node
    want, live = s["prev"].long(), torch.ones(n, dtype=torch.bool, device=DEV)
    path = torch.full((n, width), -1, dtype=torch.long, device=DEV)
    count = torch.zeros(n, dtype=torch.long, device=DEV)
    for i in range(width):
        fits = live[owner] & (parent == at[owner]) & (s["token"].long() == want[owner])
        best = torch.full((n,), nodes, dtype=torch.long, device=DEV)
        best = best.scatter_reduce(0, owner, torch.where(fits, local, nodes), "amin")
        live = best < nodes
        at = torch.where(live, best, at)
        path[:, i] = torch.where(live, best, -1)
        count += live
        want = torch.where(live, s["target"].long()[(s["first"].long()[:-1] + at).clamp(min=0)], want)
    i32 = torch.int32
    return {"path": path.to(i32), "count": count.to(i32), "next": want.to(i32)}


def _commit(s):
    pool, page = s["pool"], s["case"]["page"]
    i = torch.arange(s["path"].shape[1], device=DEV)[None, :]
    b, j = (i < s["count"][:, None]).nonzero(as_tuple=True)
    base = s["geom"][b, 1].long()
    src, dst = base + s["path"][b, j].long(), base + j
    frm = (pool["table"][b, src // page].long(), src % page)
    to = (pool["table"][b, dst // page].long(), dst % page)
    for name in ("k", "v", "ks", "vs"):
        if pool[name] is not None and not (name in ("v", "vs") and s["case"]["shared"]):
            pool[name][to] = pool[name][frm]
    return _commit_out(s)


def _commit_out(s):
    pool = s["pool"]
    if pool["ks"] is None:
        return {"k": pool["k"], "v": pool["v"]}
    f8 = torch.float8_e4m3fn
    return {"k": pool["k"].view(f8), "v": pool["v"].view(f8), "k_scale": pool["ks"], "v_scale": pool["vs"]}


_PLAIN = {"tree": _tree, "pages": _pages, "accept": _accept, "commit": _commit}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    s["step"]()
    if op == "tree":
        return {"o": s["o"], "lse": s["lse"]}
    if op == "pages":
        return _pages_out(s, s)
    if op == "accept":
        return {"path": s["path"], "count": s["count"], "next": s["next"]}
    return _commit_out(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, n = case["op"], case["n_seq"]
    if op == "pages":
        grown = 0.95 * case["new"] * 0.6 * n  # rows that get a slot, on average
        pages = grown / case["page"]
        return {"bytes": int(n * 4 * (6 + 2 * 2) + 8 * grown + 24 * pages), "flops": int(grown)}
    new = _new(case)
    if op == "accept":
        return {"bytes": 4 * (3 * sum(new) + n * (max(new) + 4)), "flops": sum(new)}
    row = D + 4 if case["fp8"] else 2 * D
    if op == "commit":
        moved = int(0.35 * sum(new))
        return {"bytes": moved * 2 * row * (1 if case["shared"] else 2) + 20 * n + 4 * moved, "flops": moved}
    rows = pairs = 0
    for (pos, n_raw, raw0, n_comp), m in zip(_geometry(case), new):
        rows += n_comp + min(WINDOW - 1, pos) + m
        if case["chain"]:
            p = pos + np.arange(m)
            pairs += int(np.minimum(n_comp, (p + 1) // case["ratio"]).sum() + np.minimum(WINDOW, p + 1).sum())
        else:
            pairs += m * (n_comp + min(WINDOW, pos + 1))  # (a window's row goes for each ancestor that comes)
    return {"bytes": rows * row * (1 if case["shared"] else 2) + sum(new) * H * (4 * D + 4), "flops": 4 * H * D * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(seg, b, n, which):
    """Rows 0 .. n-1 of sequence b, page by page."""
    if n == 0:
        return torch.zeros((0, D), dtype=torch.float64, device=DEV)
    pages = seg["table"][b, : -(-n // seg["page"])].long()
    rows = seg[which][pages].reshape(-1, D)[:n]
    if seg[which + "s"] is None:
        return rows.double()
    return rows.view(torch.float8_e4m3fn).double() * seg[which + "s"][pages].reshape(-1)[:n, None].double()


def _ancestry(parent, n):
    """Each node's way up to its root, itself first."""
    ways = []
    for t in range(n):
        up = t - 1 if parent is None else int(parent[t])
        ways.append([t] + (ways[up] if 0 <= up < t else []))
    return ways


def exact(case, seed):
    global own
    if case["op"] != "tree":
        return None  # whole numbers and moved rows: nothing is rounded
    kept_own, own = own, False
    s = prepare(case, seed)
    own = kept_own
    parents = None if s["parent"] is None else s["parent"].cpu().numpy()
    o, lse, first = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV), [], 0
    for b, ((pos, n_raw, raw0, n_comp), n) in enumerate(zip(s["geom"].tolist(), s["new"])):
        rk, rv = (_exact_rows(s["raw"], b, n_raw + n, x) for x in "kv")
        ck, cv = (_exact_rows(s["comp"], b, n_comp, x) for x in "kv")
        ways = None if parents is None else _ancestry(parents[first:first + n], n)
        for t in range(n):
            depth = t if ways is None else len(ways[t]) - 1
            p = pos + depth
            lo = min(max(0, p + 1 - WINDOW - raw0), n_raw)
            own_rows = list(range(max(0, t + 1 - WINDOW), t + 1)) if ways is None else sorted(ways[t][:WINDOW])
            pick = torch.tensor(list(range(lo, n_raw)) + [n_raw + u for u in own_rows], device=DEV)
            nc = min(n_comp, (p + 1) // case["ratio"])
            x = torch.cat([s["q"][first + t].double() @ m.T for m in (rk[pick], ck[:nc])], 1) / math.sqrt(D)
            lse.append(torch.logsumexp(x, 1))
            w = torch.softmax(x, 1)
            o[first + t] = w[:, :len(pick)] @ rv[pick] + w[:, len(pick):] @ cv[:nc]
        first += n
    return {"o": o, "lse": torch.stack(lse)}
