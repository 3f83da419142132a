"""The speculative-decoding operators: cases, inputs, plain forms and exact results.

A serving step of a model whose queries and keys come out of the projection
runs them in this order, over one paged cache:

  norm      per-head RMSNorm of q and k with the position rotation (and its gradient),
  append    the same pass over new tokens, writing K and V into the cache,
  attention every drafted node over the row's cached tokens and its own ancestors,
  verify    the drafted tree against the target's probabilities,
  cache     pages reserved, forked (copy on write), compacted to the accepted path, freed.

`run` computes an operator in plain torch operations, or, where `own` is true,
by the calls a user makes of `ulysses_qkv_proj_gb300.binding`.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # four decode requests, one new token each: pure latency
        dict(name="append_decode", op="append", n=4, nodes=1, heads=32, kv_heads=8, dim=128, rot=128,
             style="rotate_half", dtype="bf16", page=16, len_min=17, len_max=1000),
        # a training batch of two sequences, the wide projection's heads with shared K heads
        dict(name="norm_train", op="norm", B=2, S=16384, heads=64, kv_heads=8, dim=128, rot=128,
             style="rotate_half", dtype="bf16"),
        # gradient of a long ragged fp16 sequence, adjacent pairs rotated
        dict(name="norm_grad_long", op="norm_grad", B=1, S=18881, heads=56, kv_heads=14, dim=128, rot=128,
             style="interleaved", dtype="fp16"),
        # gradient of a short fine-tuning batch with half of a small head rotated
        dict(name="norm_grad_short", op="norm_grad", B=3, S=77, heads=16, kv_heads=4, dim=64, rot=32,
             style="rotate_half", dtype="bf16"),
        # one serving step's page work: rooms for the drafts, then the accepted paths pulled together
        dict(name="cache_step", op="cache_step", n=64, nodes=16, layers=8, kv_heads=8, dim=128, page=16,
             dtype="bf16", len_min=3, len_max=200),
        # prompts forked into samples, each fork taking its own copy of the open page
        dict(name="cache_fork", op="cache_fork", n=64, sources=8, layers=8, kv_heads=8, dim=128, page=64,
             dtype="bf16", len_min=65, len_max=700),
        # one request, one token: the latency of a chat turn
        dict(name="attention_single", op="attention", n=1, nodes=1, heads=32, kv_heads=8, dim=128, page=16,
             dtype="bf16", len_min=4097, len_max=4097),
        # a full decode batch of very unequal lengths
        dict(name="attention_batch", op="attention", n=64, nodes=1, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", len_min=130, len_max=32000),
        # drafted trees of 32 nodes with eight query heads to a K head
        dict(name="attention_tree", op="attention", n=16, nodes=32, heads=64, kv_heads=8, dim=128, page=32,
             dtype="bf16", len_min=900, len_max=16001),
        # wide trees over narrow fp16 heads, a page that does not divide a tile
        dict(name="attention_wide", op="attention", n=6, nodes=61, heads=16, kv_heads=16, dim=64, page=48,
             dtype="fp16", len_min=5, len_max=30011),
        # a chain of four drafted tokens for a few requests
        dict(name="verify_chain", op="verify", n=4, nodes=5, branch=1, vocab=32003, drafts=True),
        # drafted trees for a full batch over a large vocabulary
        dict(name="verify_tree", op="verify", n=48, nodes=32, branch=3, vocab=131075, drafts=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["append", "norm", "norm_grad", "cache_step", "cache_fork", "attention", "attention",
                     "attention", "verify", "verify"])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8, 8, 14])
    group = rng.choice([1, 2, 4, 7, 8])
    if op in ("norm", "norm_grad", "append"):
        case = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    style=rng.choice(["rotate_half", "interleaved"]), dtype=dtype)
        if op == "append":
            lo = spread(1, 300)
            case.update(n=spread(1, 128), nodes=spread(1, 64), page=rng.choice([16, 32, 48, 64, 128]),
                        len_min=lo, len_max=lo + spread(1, 700))
        else:
            room = 2 * 16384 * 72 * 128 // ((kv * group + kv) * dim)
            B = rng.choice([1, 2, 3])
            case.update(B=B, S=spread(5, min(20000, room // B // 2)))
        return case
    if op == "cache_step":
        lo = spread(1, 100)
        return dict(op=op, n=spread(1, 64), nodes=spread(1, 64), layers=rng.randint(1, 8), kv_heads=min(kv, 8),
                    dim=dim, page=rng.choice([16, 32, 48, 64]), dtype=dtype, len_min=lo, len_max=lo + spread(1, 100))
    if op == "cache_fork":
        lo = spread(1, 200)
        sources = rng.randint(1, 8)
        return dict(op=op, n=spread(sources, 64), sources=sources, layers=rng.randint(1, 8), kv_heads=min(kv, 8),
                    dim=dim, page=rng.choice([16, 32, 48, 64]), dtype=dtype, len_min=lo, len_max=lo + spread(1, 400))
    if op == "attention":
        n = spread(1, 64)
        top = min(40000, 64 * 6000 * 8 // (n * kv))
        lo = spread(1, max(2, top // 4))
        nodes = rng.choice([1, 1, spread(2, 64)])
        if n * kv * group * nodes > 16 * 64 * 32:
            nodes = max(1, 16 * 64 * 32 // (n * kv * group))
        return dict(op=op, n=n, nodes=nodes, heads=kv * group, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128]), dtype=dtype, len_min=lo,
                    len_max=max(lo, spread(lo, top)))
    branch = rng.choice([1, 1, 2, 4])
    vocab = spread(1000, 131075)
    nodes = spread(1, 48)
    n = max(1, min(spread(1, 64), 48 * 32 * 131075 // (vocab * nodes)))
    return dict(op=op, n=n, nodes=nodes, branch=branch, vocab=vocab, drafts=rng.random() < 0.7)


# ------------------------------------------------------------------ what a case fixes

def _lens(case, n=None):
    """The rows' lengths: spread over [len_min, len_max], in a fixed mixed order."""
    n = n or case["n"]
    lo, hi = case["len_min"], case["len_max"]
    vals = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    if n == 1:
        vals = [hi]
    random.Random(n * 1009 + lo).shuffle(vals)
    return vals


def _accepted(case):
    """Nodes each row keeps in a cache step (the root among them)."""
    most = (case["nodes"] + 1) // 2
    return [1 + (7 * i + 3) % most for i in range(case["n"])]


def _blocks(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows = case["B"] * case["S"] * (case["heads"] + case["kv_heads"])
        el = rows * case["dim"]
        table = case["S"] * case["rot"] * 4 + case["B"] * case["S"] * 4
        if op == "norm":
            return {"bytes": 2 * el * 2 + table, "flops": 8 * el}
        return {"bytes": 3 * el * 2 + table, "flops": 20 * el}
    if op == "append":
        tokens = case["n"] * case["nodes"]
        el = tokens * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * el * 2 + tokens * (case["rot"] * 4 + 4), "flops": 8 * el}
    token = 2 * case["kv_heads"] * case["dim"] * 2 if "kv_heads" in case else 0
    if op == "cache_step":
        moved = sum(k - 1 for k in _accepted(case)) * case["layers"]
        return {"bytes": 2 * moved * token + case["n"] * (case["nodes"] + 8) * 4, "flops": 0}
    if op == "cache_fork":
        src = _lens(case, case["sources"])
        copies = sum(1 for i in range(case["n"]) if src[i % case["sources"]] % case["page"])
        refs = sum(_blocks(src[i % case["sources"]], case["page"]) for i in range(case["n"]))
        return {"bytes": 2 * copies * case["page"] * case["layers"] * token + 16 * refs, "flops": 0}
    if op == "attention":
        keys = sum(L + case["nodes"] for L in _lens(case))
        q = case["n"] * case["nodes"] * case["heads"] * case["dim"]
        return {"bytes": keys * token + 2 * q * 2 + q // case["dim"] * 4,
                "flops": 4 * keys * case["nodes"] * case["heads"] * case["dim"]}
    # verify: at the least the row that the next token is drawn from, with its draft's
    return {"bytes": case["n"] * case["vocab"] * 4 * (2 if case["drafts"] else 1), "flops": 3 * case["n"] * case["vocab"]}


# ------------------------------------------------------------------ inputs

def _angles(positions, rot):
    half = rot // 2
    f = 1e4 ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _tree(rng, nodes, branch):
    """Parents of a tree in the order a drafter emits it: every parent before its
    children, at most `branch` children to a node; node 0 is the last emitted token."""
    parents, room = [-1], {0: branch}
    for i in range(1, nodes):
        p = rng.choice(sorted(room)[-(2 * branch + 1):])
        parents.append(p)
        room[p] -= 1
        if room[p] == 0:
            del room[p]
        room[i] = branch
    return parents


def _ancestors(parents):
    masks = []
    for i, p in enumerate(parents):
        m = (masks[p] if p >= 0 else 0) | (1 << i)
        masks.append(m)
    return [m - (1 << 64) if m >> 63 else m for m in masks]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _pool(gen, case, pages, layers):
    shape = (layers, pages, case["kv_heads"], case["page"], case["dim"])
    dt = DTYPES[case["dtype"]]
    return [torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(2)]


def _cache(gen, case, lens, rows, layers, room, spare):
    """A cache whose first len(lens) rows hold tokens, with `room` more reserved in each."""
    page = case["page"]
    width = max(_blocks(L + max(room, case.get("nodes", 1)), page) for L in lens) + 1
    need = [_blocks(L + room, page) for L in lens]
    pages = sum(need) + spare
    order = list(range(pages))
    random.Random(sum(lens) + pages).shuffle(order)
    table = torch.full((rows, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for r, b in enumerate(need):
        ids = torch.tensor(order[at:at + b], dtype=torch.int32)
        table[r, :b] = ids
        refs[ids.long()] = 1
        at += b
    k, v = _pool(gen, case, pages, layers)
    full = list(lens) + [0] * (rows - len(lens))
    return dict(kpool=k, vpool=v, table=table.cuda(), refs=refs.cuda(), lens=_i32(full), page=page, host_lens=full)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from ulysses_qkv_proj_gb300 import binding as qb
        if "kpool" in st:
            st["cache"] = qb.PagedCache(st["kpool"], st["vpool"], st["table"], st["lens"], st["refs"])
        if case["op"] == "norm_grad":
            st["workspace"] = qb.qk_norm_rope_workspace(st["q"], st["k"])
        if case["op"] == "attention":
            st["workspace"] = qb.tree_attention_workspace(st["q"], st["cache"])
    return st


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    rng = random.Random(seed * 31 + 5)
    op = case["op"]
    st = {"case": case}
    if op in ("norm", "norm_grad", "append"):
        dt, D = DTYPES[case["dtype"]], case["dim"]
        Hq, Hk = case["heads"], case["kv_heads"]
        B, S = (case["n"], case["nodes"]) if op == "append" else (case["B"], case["S"])
        proj = torch.randn((B, S, Hq + 2 * Hk, D), generator=gen, device="cuda", dtype=dt)
        st.update(q=proj[:, :, :Hq], k=proj[:, :, Hq:Hq + Hk], v=proj[:, :, Hq + Hk:])
        for name in ("qw", "kw"):
            st[name] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        if op == "append":
            lens = _lens(case)
            st.update(_cache(gen, case, lens, case["n"], 1, S, 3))
            st["rows"] = _i32(list(range(case["n"])))
            depth = []
            for L in lens:
                d = []
                for p in _tree(rng, S, 3):
                    d.append(0 if p < 0 else d[p] + 1)
                depth.append([L + x for x in d])
            st["positions"] = _i32(depth)
            st["angles"] = _angles(max(lens) + S, case["rot"])
        else:
            st["positions"] = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, S).contiguous()
            st["angles"] = _angles(S, case["rot"])
            st["k_out"] = torch.empty((B, S, Hk, D), device="cuda", dtype=dt)
        st["q_out"] = torch.empty((B, S, Hq, D), device="cuda", dtype=dt)
        if op == "norm_grad":
            st["gq"] = torch.randn((B, S, Hq, D), generator=gen, device="cuda", dtype=dt)
            st["gk"] = torch.randn((B, S, Hk, D), generator=gen, device="cuda", dtype=dt)
            st["gqw"], st["gkw"] = (torch.empty(D, device="cuda") for _ in range(2))
        return st
    if op == "cache_step":
        lens, kept = _lens(case), _accepted(case)
        st.update(_cache(gen, case, lens, case["n"], case["layers"], 0, case["n"] * (_blocks(case["nodes"], case["page"]) + 1)))
        path = torch.full((case["n"], case["nodes"]), -1, dtype=torch.int32)
        for i, c in enumerate(kept):
            path[i, :c] = torch.tensor([0] + sorted(rng.sample(range(c, case["nodes"]), c - 1)), dtype=torch.int32)
        st.update(rows=_i32(list(range(case["n"]))), base=_i32(lens), room=_i32([case["nodes"]] * case["n"]),
                  path=path.cuda(), kept=_i32(kept))
        return st
    if op == "cache_fork":
        src = _lens(case, case["sources"])
        n, s = case["n"], case["sources"]
        st.update(_cache(gen, case, src, s + n, case["layers"], 0, 2 * n))
        st.update(src=_i32([i % s for i in range(n)]), dst=_i32([s + i for i in range(n)]),
                  zeros=_i32([0] * n), room=_i32([1] * n))
        return st
    if op == "attention":
        lens, N = _lens(case), case["nodes"]
        st.update(_cache(gen, case, lens, case["n"], 1, N, 1))
        dt = DTYPES[case["dtype"]]
        shape = (case["n"], N, case["heads"], case["dim"])
        st["q"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        st["masks"] = torch.tensor([_ancestors(_tree(rng, N, 3)) for _ in lens], dtype=torch.int64).cuda()
        st["rows"] = _i32(list(range(case["n"])))
        st["out"] = torch.empty(shape, device="cuda", dtype=dt)
        st["lse"] = torch.empty(shape[:3], device="cuda")
        return st
    n, N, V = case["n"], case["nodes"], case["vocab"]
    base = torch.randn((n, N, V), generator=gen, device="cuda")
    target = torch.softmax(base * 2.5, -1)
    trees = [_tree(rng, N, case["branch"]) for _ in range(n)]
    parents = torch.tensor(trees, dtype=torch.int32).cuda()
    above = parents.clamp(min=0).long()
    if case["drafts"]:
        # the drafter sees the same text: its distribution is a blurred target
        base.mul_(2.0).add_(torch.randn((n, N, V), generator=gen, device="cuda"))
        draft = torch.softmax(base, -1)
    else:
        draft = None
    del base
    from_q = draft if draft is not None else target
    pick = torch.rand((n, N), generator=gen, device="cuda", dtype=torch.float64)
    tokens = torch.empty((n, N), dtype=torch.int32, device="cuda")
    for i in range(N):
        row = from_q[torch.arange(n, device="cuda"), above[:, i]].double().cumsum(-1)
        tokens[:, i] = torch.searchsorted(row, (pick[:, i:i + 1] * row[:, -1:]), right=True)[:, 0].clamp(max=V - 1).int()
    st.update(target=target, draft=draft, parents=parents, tokens=tokens,
              accept=torch.rand((n, N), generator=gen, device="cuda"), sample=torch.rand(n, generator=gen, device="cuda"),
              path=torch.empty((n, N), dtype=torch.int32, device="cuda"),
              kept=torch.empty(n, dtype=torch.int32, device="cuda"), next=torch.empty(n, dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    from ulysses_qkv_proj_gb300 import binding as qb
    case = st["case"]
    op = case["op"]
    if op == "norm":
        qb.qnre_qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["angles"], st["positions"], st["q_out"],
                             st["k_out"], rope_style=case["style"])
        return st["q_out"], st["k_out"]
    if op == "norm_grad":
        gq, gk = torch.empty_like(st["gq"]), torch.empty_like(st["gk"])
        qb.qnre_qk_norm_rope_backward(st["gq"], st["gk"], st["q"], st["k"], st["qw"], st["kw"], st["angles"],
                                      st["positions"], gq, gk, st["gqw"], st["gkw"], st["workspace"],
                                      rope_style=case["style"])
        return gq, gk, st["gqw"], st["gkw"]
    if op == "append":
        qb.qnre_qkv_norm_rope_append(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["angles"], st["positions"],
                                     st["q_out"], st["cache"], 0, st["rows"], rope_style=case["style"])
        return st["q_out"], st["kpool"], st["vpool"]
    if op == "cache_step":
        qb.qnre_cache_truncate(st["cache"], st["rows"], st["base"])
        qb.qnre_cache_reserve(st["cache"], st["rows"], st["room"])
        qb.qnre_cache_compact(st["cache"], st["rows"], st["path"], st["kept"])
        return st["kpool"], st["vpool"], st["table"], st["refs"], st["lens"]
    if op == "cache_fork":
        qb.qnre_cache_truncate(st["cache"], st["dst"], st["zeros"])
        qb.qnre_cache_fork(st["cache"], st["src"], st["dst"])
        qb.qnre_cache_reserve(st["cache"], st["dst"], st["room"])
        return st["kpool"], st["vpool"], st["table"], st["refs"], st["lens"]
    if op == "attention":
        qb.qnre_tree_attention(st["q"], st["cache"], 0, st["rows"], st["masks"], st["out"], lse=st["lse"],
                               workspace=st["workspace"])
        return st["out"], st["lse"]
    qb.qnre_verify_tree(st["target"], st["draft"], st["tokens"], st["parents"], st["accept"], st["sample"],
                        st["path"], st["kept"], st["next"])
    return st["path"], st["kept"], st["next"]


# ------------------------------------------------------------------ the plain forms

def _rotate(x, c, s, style, back=False):
    """x [..., D] in 32 bits, c and s [..., 1, rot/2]; the transpose where `back`."""
    half = c.shape[-1]
    if back:
        s = -s
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if style == "rotate_half":
        a, b = r[..., :half], r[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _norm_rope(x, w, c, s, style):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, c, s, style).to(x.dtype)


def _norm_rope_grad(g, x, w, c, s, style):
    y = x.float()
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    hat = y * r
    n = _rotate(g.float(), c, s, style, back=True)
    gw = (n * hat).double().sum((0, 1, 2)).float()
    t = n * w.float()
    return (r * (t - hat * (t * hat).mean(-1, keepdim=True))).to(x.dtype), gw


def _truncate(st, rows, lens):
    rows = rows.long()
    table, page = st["table"], st["page"]
    j = torch.arange(table.shape[1], device="cuda")
    entry = table[rows]
    drop = (j[None] >= ((lens + page - 1) // page)[:, None]) & (entry >= 0)
    st["refs"].scatter_add_(0, entry.clamp(min=0).flatten().long(), -drop.flatten().int())
    table[rows] = torch.where(drop, -1, entry)
    st["lens"][rows] = torch.minimum(st["lens"][rows], lens)


def _fork(st, src, dst):
    table, page = st["table"], st["page"]
    lens = st["lens"][src.long()]
    j = torch.arange(table.shape[1], device="cuda")
    entry = torch.where(j[None] < ((lens + page - 1) // page)[:, None], table[src.long()], -1)
    st["refs"].scatter_add_(0, entry.clamp(min=0).flatten().long(), (entry >= 0).flatten().int())
    table[dst.long()] = entry
    st["lens"][dst.long()] = lens


def _reserve(st, rows, room):
    rows = rows.long()
    table, refs, page = st["table"], st["refs"], st["page"]
    lens = st["lens"][rows]
    j = torch.arange(table.shape[1], device="cuda")[None]
    entry = table[rows]
    window = (j >= (lens // page)[:, None]) & (j < ((lens + room + page - 1) // page)[:, None])
    shared = window & (entry >= 0) & (refs[entry.clamp(min=0).long()] > 1)
    need = (window & (entry < 0)) | shared
    free = torch.argsort(refs != 0, stable=True).int()      # free pages, lowest first
    ids = free[(need.flatten().int().cumsum(0) - 1).clamp(min=0).long()].view_as(entry)
    copied = shared & (j * page < lens[:, None])
    source, target = entry[copied].long(), ids[copied].long()
    for pool in (st["kpool"], st["vpool"]):
        pool[:, target] = pool[:, source]
    refs.scatter_add_(0, entry.clamp(min=0).flatten().long(), -shared.flatten().int())
    refs[ids[need].long()] = 1
    table[rows] = torch.where(need, ids, entry)


def _compact(st, rows, path, kept):
    rows = rows.long()
    page = st["page"]
    lens = st["lens"][rows]
    j = torch.arange(path.shape[1], device="cuda")[None]
    use = j < kept[:, None]
    from_at = lens[:, None] + path.clamp(min=0)
    to_at = lens[:, None] + j.int()
    entry = st["table"][rows]
    last = entry.shape[1] - 1
    sp = entry.gather(1, (from_at // page).clamp(max=last).long())[use].long()
    tp = entry.gather(1, (to_at // page).clamp(max=last).long())[use].long()
    ss, ts = (from_at % page)[use].long(), (to_at % page)[use].long()
    for pool in (st["kpool"], st["vpool"]):
        pool[:, tp, :, ts] = pool[:, sp, :, ss]
    st["lens"][rows] = lens + kept
    _truncate(st, rows.int(), lens + kept)


def _attention(st):
    case = st["case"]
    n, N, Hq, D = st["q"].shape
    Hk, page = case["kv_heads"], st["page"]
    G = Hq // Hk
    out = torch.empty_like(st["q"])
    lse = torch.empty((n, N, Hq), device="cuda")
    bits = torch.arange(N, device="cuda")
    for i in range(n):
        L = st["host_lens"][i]
        blocks = _blocks(L + N, page)
        ids = st["table"][i, :blocks].long()
        k = st["kpool"][0, ids].transpose(0, 1).reshape(Hk, blocks * page, D)[:, :L + N].float()
        v = st["vpool"][0, ids].transpose(0, 1).reshape(Hk, blocks * page, D)[:, :L + N].float()
        q = st["q"][i].float().view(N, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * N, D)
        s = (q @ k.transpose(1, 2)).view(Hk, G, N, L + N) * (1 / math.sqrt(D))
        see = (st["masks"][i][:, None] >> bits[None]) & 1
        s[..., L:].masked_fill_(see == 0, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        o = (p / z).view(Hk, G * N, L + N) @ v
        out[i] = o.view(Hk, G, N, D).permute(2, 0, 1, 3).reshape(N, Hq, D).to(out.dtype)
        lse[i] = (m + torch.log(z))[..., 0].permute(2, 0, 1).reshape(N, Hq)
    return out, lse


def _verify(st):
    """The tree walked node by node for the whole batch: at the node reached, its
    children are tried in order against p_i = max(p - a q, 0) / R, where a rejection
    takes a to a + R and R to the sum that is left (without draft probabilities each
    child stands for itself: a rejection takes its token out of p)."""
    target, draft, tokens, parents = st["target"], st["draft"], st["tokens"], st["parents"]
    n, N, V = target.shape
    at = torch.arange(n, device="cuda")
    cur = torch.zeros(n, dtype=torch.long, device="cuda")
    a = torch.zeros(n, dtype=torch.float64, device="cuda")
    R = torch.ones(n, dtype=torch.float64, device="cuda")
    path = torch.full((n, N), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    kept = torch.ones(n, dtype=torch.long, device="cuda")
    p = target[:, 0].double()
    q = draft[:, 0].double() if draft is not None else None
    left = p
    for i in range(1, N):
        child = parents[:, i] == cur
        x = tokens[:, i].long()
        u = st["accept"][:, i].double()
        qx = q[at, x] if q is not None else 1.0
        good = child & (u * qx * R < left[at, x])
        bad = child & ~good
        if q is not None:
            a = torch.where(bad, a + R, a)
            tried = torch.clamp(p - a[:, None] * q, min=0)
            R = torch.where(bad, tried.sum(-1), R)
            left = torch.where(bad[:, None], tried, left)
        else:
            R = torch.where(bad, R - left[at, x], R)
            left = left.clone()
            left[at, x] = torch.where(bad, 0.0, left[at, x])
        path[at, kept.clamp(max=N - 1)] = torch.where(good, i, path[at, kept.clamp(max=N - 1)])
        kept = kept + good.long()
        cur = torch.where(good, i, cur)
        a = torch.where(good, 0.0, a)
        R = torch.where(good, 1.0, R)
        p = torch.where(good[:, None], target[:, i].double(), p)
        if q is not None:
            q = torch.where(good[:, None], draft[:, i].double(), q)
        left = torch.where(good[:, None], p, left)
    left = torch.where((left.sum(-1) > 0)[:, None], left, p)
    c = left.cumsum(-1)
    t = st["sample"].double() * c[:, -1]
    following = torch.searchsorted(c, t[:, None], right=True)[:, 0]
    last = V - 1 - (left.flip(-1) > 0).int().argmax(-1)
    return path, kept.int(), torch.minimum(following, last).int()


def run(state):
    if own:
        return _run_own(state)
    st, case = state, state["case"]
    op = case["op"]
    if op in ("norm", "norm_grad", "append"):
        row = st["angles"][st["positions"].long()][:, :, None]
        half = case["rot"] // 2
        c, s = row[..., :half], row[..., half:]
    if op == "norm":
        return (_norm_rope(st["q"], st["qw"], c, s, case["style"]), _norm_rope(st["k"], st["kw"], c, s, case["style"]))
    if op == "norm_grad":
        gq, gqw = _norm_rope_grad(st["gq"], st["q"], st["qw"], c, s, case["style"])
        gk, gkw = _norm_rope_grad(st["gk"], st["k"], st["kw"], c, s, case["style"])
        return gq, gk, gqw, gkw
    if op == "append":
        q = _norm_rope(st["q"], st["qw"], c, s, case["style"])
        k = _norm_rope(st["k"], st["kw"], c, s, case["style"])
        at = st["lens"][st["rows"].long()][:, None] + torch.arange(case["nodes"], device="cuda")[None]
        page = st["table"][st["rows"].long()].gather(1, at // st["page"]).long()
        slot = at % st["page"]
        st["kpool"][0, page, :, slot] = k
        st["vpool"][0, page, :, slot] = st["v"]
        return q, st["kpool"], st["vpool"]
    if op == "cache_step":
        _truncate(st, st["rows"], st["base"])
        _reserve(st, st["rows"], st["room"])
        _compact(st, st["rows"], st["path"], st["kept"])
        return st["kpool"], st["vpool"], st["table"], st["refs"], st["lens"]
    if op == "cache_fork":
        _truncate(st, st["dst"], st["zeros"])
        _fork(st, st["src"], st["dst"])
        _reserve(st, st["dst"], st["room"])
        return st["kpool"], st["vpool"], st["table"], st["refs"], st["lens"]
    if op == "attention":
        return _attention(st)
    return _verify(st)


# ------------------------------------------------------------------ exact results

def _turn(x, w, angles, style):
    """The norm and the rotation in 64 bits, each pair as one complex number."""
    half = angles.shape[-1] // 2
    z = torch.complex(angles[..., :half], angles[..., half:])[:, :, None]
    y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
    lead, rest = y[..., :2 * half], y[..., 2 * half:]
    if style == "rotate_half":
        t = torch.complex(lead[..., :half], lead[..., half:]) * z
        return torch.cat([t.real, t.imag, rest], -1)
    t = torch.view_as_complex(lead.unflatten(-1, (half, 2)).contiguous()) * z
    return torch.cat([torch.view_as_real(t).flatten(-2), rest], -1)


class _Pages:
    """The cache's bookkeeping on lists, one row and one page at a time."""

    def __init__(self, st):
        self.page = st["page"]
        self.table, self.refs, self.lens = st["table"].tolist(), st["refs"].tolist(), st["lens"].tolist()
        self.pools = st["kpool"], st["vpool"]

    def truncate(self, rows, lens):
        for r, length in zip(rows, lens):
            for j, e in enumerate(self.table[r]):
                if e >= 0 and j * self.page >= length:
                    self.refs[e] -= 1
                    self.table[r][j] = -1
            self.lens[r] = min(self.lens[r], length)

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            for j in range(_blocks(self.lens[s], self.page)):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            self.lens[d] = self.lens[s]

    def reserve(self, rows, room):
        shared = [c > 1 for c in self.refs]
        free = iter([i for i, c in enumerate(self.refs) if c == 0])
        for r, more in zip(rows, room):
            length = self.lens[r]
            for j in range(length // self.page, _blocks(length + more, self.page)):
                e = self.table[r][j]
                if e >= 0 and not shared[e]:
                    continue
                new = next(free)
                if e >= 0:
                    self.refs[e] -= 1
                    if j * self.page < length:
                        for pool in self.pools:
                            pool[:, new] = pool[:, e]
                self.table[r][j] = new
                self.refs[new] = 1

    def compact(self, rows, path, kept):
        for r, nodes, count in zip(rows, path, kept):
            length = self.lens[r]
            for j in range(count):
                a, b = length + nodes[j], length + j
                for pool in self.pools if a != b else ():
                    pool[:, self.table[r][b // self.page], :, b % self.page] = \
                        pool[:, self.table[r][a // self.page], :, a % self.page]
            self.lens[r] = length + count
            self.truncate([r], [length + count])

    def result(self):
        as_i32 = [torch.tensor(x, dtype=torch.int32) for x in (self.table, self.refs, self.lens)]
        return (*self.pools, *as_i32)


def _exact_attention(st):
    case, page = st["case"], st["page"]
    n, N, Hq, D = st["q"].shape
    G = Hq // case["kv_heads"]
    out = torch.zeros((n, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, N, Hq), dtype=torch.float64, device="cuda")
    for i, L in enumerate(st["host_lens"]):
        at = torch.arange(L + N, device="cuda")
        pages = st["table"][i].long()[at // page]
        node = torch.arange(N, device="cuda")
        hidden = torch.cat([torch.zeros((N, L), dtype=torch.bool, device="cuda"),
                            torch.bitwise_right_shift(st["masks"][i][:, None], node[None]) % 2 == 0], 1)
        for h in range(case["kv_heads"]):
            k = st["kpool"][0][pages, h, at % page].double()
            v = st["vpool"][0][pages, h, at % page].double()
            s = torch.einsum("tgd,ld->gtl", st["q"][i, :, h * G:(h + 1) * G].double(), k) / D ** 0.5
            s = torch.where(hidden[None], -math.inf, s)
            z = torch.logsumexp(s, -1)
            out[i, :, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", torch.exp(s - z[..., None]), v)
            lse[i, :, h * G:(h + 1) * G] = z.t()
    return out, lse


def _exact_verify(st):
    tokens, parents = st["tokens"].tolist(), st["parents"].tolist()
    accept, sample = st["accept"].double().tolist(), st["sample"].double().tolist()
    paths, counts, following = [], [], []
    for b, (toks, up) in enumerate(zip(tokens, parents)):
        def rows(node):
            q = st["draft"][b, node].double() if st["draft"] is not None else None
            return st["target"][b, node].double(), q

        node, path = 0, [0]
        p, q = rows(0)
        while True:
            dist, reached = p, None
            for child in [i for i in range(1, len(up)) if up[i] == node]:
                x = toks[child]
                px, qx = dist[x].item(), q[x].item() if q is not None else 1.0
                if accept[b][child] * qx < px:
                    reached = child
                    break
                if q is not None:
                    dist = (dist - q).clamp(min=0)
                else:
                    dist = dist.clone()
                    dist[x] = 0
                if q is not None:
                    dist = dist / dist.sum()
                else:
                    # the token's own mass leaves; the rest is one less it
                    dist = dist / (1 - px)
            if reached is None:
                break
            node = reached
            path.append(node)
            p, q = rows(node)
        dist = dist if dist.sum() > 0 else p
        c = dist.cumsum(0)
        pick = int((c <= sample[b] * c[-1]).sum())
        following.append(min(pick, int(dist.nonzero().max())))
        paths.append(path + [-1] * (len(up) - len(path)))
        counts.append(len(path))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (paths, counts, following))


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad", "append"):
        angles = st["angles"].double()[st["positions"].long()]
    if op == "norm":
        return tuple(_turn(st[x].double(), st[x + "w"].double(), angles, case["style"]) for x in "qk")
    if op == "norm_grad":
        rows, weights = [], []
        for x in "qk":
            leaf = st[x].double().requires_grad_()
            w = st[x + "w"].double().requires_grad_()
            gx, gw = torch.autograd.grad(_turn(leaf, w, angles, case["style"]), (leaf, w), st["g" + x].double())
            rows.append(gx)
            weights.append(gw)
        return (*rows, *weights)
    if op == "append":
        q, k = (_turn(st[x].double(), st[x + "w"].double(), angles, case["style"]) for x in "qk")
        pools = st["kpool"].double(), st["vpool"].double()
        table = st["table"].tolist()
        for i, L in enumerate(st["host_lens"]):
            for j in range(case["nodes"]):
                page, slot = table[i][(L + j) // st["page"]], (L + j) % st["page"]
                pools[0][0, page, :, slot] = k[i, j]
                pools[1][0, page, :, slot] = st["v"][i, j].double()
        return (q, *pools)
    if op == "cache_step":
        pages = _Pages(st)
        rows = st["rows"].tolist()
        pages.truncate(rows, st["base"].tolist())
        pages.reserve(rows, st["room"].tolist())
        pages.compact(rows, st["path"].tolist(), st["kept"].tolist())
        return pages.result()
    if op == "cache_fork":
        pages = _Pages(st)
        dst = st["dst"].tolist()
        pages.truncate(dst, st["zeros"].tolist())
        pages.fork(st["src"].tolist(), dst)
        pages.reserve(dst, st["room"].tolist())
        return pages.result()
    if op == "attention":
        return _exact_attention(st)
    return _exact_verify(st)
