"""Operators for many answers from shared prompts: cases, inputs, plain forms and exact results.

A server that draws several samples from a prompt, or whose requests begin with
the same long text, runs these beside the cache's own calls:

  table      the cos/sin table of plain or scaled rotary positions,
  attention  rows whose leading pages are the same read them once for the group; scores may
             be capped by a tanh and get a bias that falls with distance,
  sample     tokens from logits with temperature, top-k, top-p and min-p and given random numbers,
  filter     the same filter as probabilities, which the verification of drafted trees takes.

`run` computes an operator in plain torch operations, or, where `own` is true,
by the calls a user makes of `ulysses_qkv_proj_gb300.binding`.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the table of a short-context model, made when a server starts or a test begins
        dict(name="table_short", op="table", n_pos=2048, rot=64, scaling="none"),
        # half a million positions of a model stretched past the length that it was trained on
        dict(name="table_long", op="table", n_pos=524288, rot=128, scaling="yarn"),
        # eight samples of one prompt: the latency of a chat turn with alternatives
        dict(name="prefix_chat", op="attention", n=8, groups=1, nodes=1, heads=32, kv_heads=8, dim=128, page=16,
             dtype="bf16", pre_min=2011, pre_max=2011, suf_min=3, suf_max=400, cap=0.0, slopes=False),
        # a full batch over a few long prompts, groups of unequal size
        dict(name="prefix_batch", op="attention", n=128, groups=6, nodes=1, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", pre_min=1500, pre_max=30011, suf_min=1, suf_max=900, cap=0.0, slopes=False),
        # capped scores over narrow fp16 heads with a K head each, a page that does not divide a tile
        dict(name="prefix_capped", op="attention", n=48, groups=3, nodes=1, heads=16, kv_heads=16, dim=64, page=48,
             dtype="fp16", pre_min=700, pre_max=16001, suf_min=5, suf_max=3000, cap=30.0, slopes=False),
        # drafts of eight nodes for the samples of two prompts, positions only by the distance bias
        dict(name="prefix_drafts", op="attention", n=24, groups=2, nodes=8, heads=56, kv_heads=14, dim=128, page=32,
             dtype="bf16", pre_min=4000, pre_max=9001, suf_min=20, suf_max=700, cap=50.0, slopes=True),
        # one request, temperature alone
        dict(name="sample_one", op="sample", n=1, vocab=32003, dtype="fp32", setting="plain"),
        # a decode batch whose requests each bring their own settings, over a large vocabulary
        dict(name="sample_mixed", op="sample", n=64, vocab=131075, dtype="fp32", setting="mixed"),
        # top-p over 16-bit logits, full of ties
        dict(name="sample_nucleus", op="sample", n=256, vocab=131075, dtype="bf16", setting="nucleus"),
        # the target's probabilities for four chains of four drafts
        dict(name="filter_chain", op="filter", n=4, nodes=5, vocab=32003, dtype="fp32", setting="top_k"),
        # the same for a full batch of trees, each request with its own settings
        dict(name="filter_tree", op="filter", n=32, nodes=32, vocab=131075, dtype="bf16", setting="mixed"),
    ]


SETTINGS = ["plain", "top_k", "nucleus", "min_p", "mixed", "greedy"]


def draw(rng):
    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["table", "attention", "attention", "attention", "sample", "sample", "filter"])
    if op == "table":
        rot = rng.choice([16, 32, 64, 96, 128, 128])
        return dict(op=op, n_pos=spread(5, 524288), rot=rot, scaling=rng.choice(["none", "linear", "base", "yarn", "wavelength"]))
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8, 8, 14])
        heads = kv * rng.choice([1, 2, 4, 7, 8])
        nodes = rng.choice([1, 1, 1, spread(2, 32)])
        n = spread(2, 128)
        top = max(40, min(30011, 128 * 64 * 12000 // (n * nodes * heads)))
        lo = spread(1, max(2, top // 2))
        suf = spread(1, 100)
        return dict(op=op, n=n, groups=spread(1, max(1, n // 2)), nodes=nodes, heads=heads, kv_heads=kv,
                    dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 48, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), pre_min=lo, pre_max=spread(lo, max(lo, top)), suf_min=suf,
                    suf_max=spread(suf, max(suf, min(3000, top))), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    slopes=rng.random() < 0.3)
    vocab = spread(1000, 131075)
    dtype = rng.choice(["fp32", "fp32", "bf16", "fp16"])
    setting = rng.choice(SETTINGS)
    if op == "sample":
        return dict(op=op, n=spread(1, 256), vocab=vocab, dtype=dtype, setting=setting)
    n, nodes = spread(1, 32), spread(1, 32)
    if dtype == "fp32":
        nodes = max(1, nodes // 2)
    return dict(op=op, n=n, nodes=nodes, vocab=vocab, dtype=dtype, setting=setting)


# ------------------------------------------------------------------ what a case fixes

def _between(lo, hi, n, salt):
    """n lengths spread over [lo, hi] in a fixed mixed order."""
    vals = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    if n == 1:
        vals = [hi]
    random.Random(n * 1009 + lo + salt).shuffle(vals)
    return vals


def _members(case):
    """Rows of each group: one at least, the rest dealt out unevenly."""
    n, g = case["n"], case["groups"]
    rng = random.Random(n * 31 + g)
    sizes = [1] * g
    for _ in range(n - g):
        sizes[min(int(rng.random() ** 1.5 * g), g - 1)] += 1
    return sizes


def _prefixes(case):
    return _between(case["pre_min"], case["pre_max"], case["groups"], 1)


def _suffixes(case):
    return _between(case["suf_min"], case["suf_max"], case["n"], 2)


def _blocks(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": case["n_pos"] * case["rot"] * 4, "flops": 16 * case["n_pos"] * case["rot"]}
    if op == "attention":
        token = 2 * case["kv_heads"] * case["dim"] * 2
        sizes, pre, suf = _members(case), _prefixes(case), _suffixes(case)
        once = sum(p // case["page"] * case["page"] if s > 1 else 0 for s, p in zip(sizes, pre))
        keys = sum(s * p for s, p in zip(sizes, pre)) + sum(suf) + case["n"] * case["nodes"]
        apart = sum(s * (p % case["page"] if s > 1 else p) for s, p in zip(sizes, pre)) + sum(suf) + case["n"] * case["nodes"]
        q = case["n"] * case["nodes"] * case["heads"] * case["dim"]
        return {"bytes": (once + apart) * token + 2 * q * 2 + q // case["dim"] * 4,
                "flops": 4 * keys * case["nodes"] * case["heads"] * case["dim"]}
    size = 4 if case["dtype"] == "fp32" else 2
    cells = case["n"] * case.get("nodes", 1) * case["vocab"]
    return {"bytes": cells * (size + (4 if op == "filter" else 0)), "flops": 4 * cells}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _tree(rng, nodes):
    """Parents of a drafted tree, every parent before its children; node 0 is the last emitted token."""
    return [-1] + [rng.randrange(max(0, i - 3), i) for i in range(1, nodes)]


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] == "attention":
        from ulysses_qkv_proj_gb300 import binding as qb
        st["cache"] = qb.PagedCache(st["kpool"], st["vpool"], st["table"], st["lens"], st["refs"])
        st["workspace"] = qb.prefix_attention_workspace(st["q"], st["cache"])
    return st


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    rng = random.Random(seed * 37 + 11)
    op = case["op"]
    st = {"case": case}
    if op == "table":
        st.update(theta=rng.choice([1e4, 5e5, 1e6]), first=rng.randrange(0, 100000), factor=rng.choice([2.0, 4.0, 8.0]),
                  original=rng.choice([4096, 8192]), out=torch.empty((case["n_pos"], case["rot"]), device="cuda"))
        return st
    if op == "attention":
        return _attention_inputs(case, st, gen, rng)
    n, N, V = case["n"], case.get("nodes", 1), case["vocab"]
    dt = DTYPES[case["dtype"]]
    # logits of a language model: a wide bell, its spread different for each request, with a few tokens far above
    sharp = 1.5 + 2.0 * torch.rand((n, 1, 1), generator=gen, device="cuda")
    logits = torch.empty((n, N, V), device="cuda", dtype=dt)
    for i in range(n):
        x = torch.randn((N, V), generator=gen, device="cuda") * sharp[i]
        at = torch.randint(0, V, (N, 12), generator=gen, device="cuda")
        x.scatter_add_(1, at, torch.rand((N, 12), generator=gen, device="cuda") * 3 * sharp[i])
        logits[i] = x.to(dt)
    kinds = {"plain": [0], "top_k": [1], "nucleus": [2], "min_p": [3], "greedy": [5], "mixed": [4, 1, 2, 0, 3, 5, 2, 4]}
    T, k, p, m = [], [], [], []
    for i in range(n):
        kind = kinds[case["setting"]][i % len(kinds[case["setting"]])]
        T.append(0.0 if kind == 5 else rng.choice([0.6, 0.7, 0.8, 1.0, 1.3]))
        k.append(rng.choice([20, 40, 50, 200, 1000]) if kind in (1, 4) else 0)
        p.append(rng.choice([0.5, 0.8, 0.9, 0.95, 0.99]) if kind in (2, 4) else 1.0)
        m.append(rng.choice([0.02, 0.05, 0.1]) if kind in (3, 4) else 0.0)
    st.update(logits=logits, temperature=torch.tensor(T).cuda(), top_k=_i32(k), top_p=torch.tensor(p).cuda(),
              min_p=torch.tensor(m).cuda())
    if op == "sample":
        st["logits"] = logits[:, 0]
        st["u"] = torch.rand(n, generator=gen, device="cuda")
        st["tokens"] = torch.empty(n, dtype=torch.int32, device="cuda")
    else:
        st["probs"] = torch.empty((n, N, V), device="cuda")
    return st


def _attention_inputs(case, st, gen, rng):
    """A cache whose rows begin with their group's prompt: its whole pages are the group's, the rest of it the row's own."""
    n, N, page, D, Hk = case["n"], case["nodes"], case["page"], case["dim"], case["kv_heads"]
    sizes, prefixes, suffixes = _members(case), _prefixes(case), _suffixes(case)
    starts = [sum(sizes[:g]) for g in range(len(sizes) + 1)]
    group = [g for g, s in enumerate(sizes) for _ in range(s)]
    lens = [prefixes[g] + s for g, s in zip(group, suffixes)]
    width = max(_blocks(L + N, page) for L in lens) + 1
    common = [p // page for p in prefixes]
    pages = sum(common) + sum(_blocks(L + N, page) - common[g] for g, L in zip(group, lens)) + 1
    order = list(range(pages))
    random.Random(pages + sum(lens)).shuffle(order)
    order = torch.tensor(order, dtype=torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    rows = list(range(n))
    random.Random(n).shuffle(rows)
    at = 0
    for g in range(len(sizes)):
        ids = order[at:at + common[g]]
        at += common[g]
        refs[ids.long()] = sizes[g]
        for i in range(starts[g], starts[g + 1]):
            more = _blocks(lens[i] + N, page) - common[g]
            mine = order[at:at + more]
            at += more
            refs[mine.long()] = 1
            table[rows[i], :common[g] + more] = torch.cat([ids, mine])
    dt = DTYPES[case["dtype"]]
    shape = (1, pages, Hk, page, D)
    row_lens = [0] * n
    for r, L in zip(rows, lens):
        row_lens[r] = L
    trees = [_tree(rng, N) for _ in range(n)]
    masks, depths = [], []
    for parents in trees:
        m, d = [], []
        for j, p in enumerate(parents):
            m.append((m[p] if p >= 0 else 0) | 1 << j)
            d.append(d[p] + 1 if p >= 0 else 0)
        masks.append(m)
        depths.append(d)
    st.update(kpool=torch.randn(shape, generator=gen, device="cuda", dtype=dt),
              vpool=torch.randn(shape, generator=gen, device="cuda", dtype=dt),
              table=table.cuda(), refs=refs.cuda(), lens=_i32(row_lens), rows=_i32(rows), groups=_i32(starts),
              host_lens=lens, host_rows=rows, host_starts=starts,
              masks=torch.tensor(masks, dtype=torch.int64).cuda(), depths=_i32(depths),
              shared=torch.empty(len(sizes), dtype=torch.int32, device="cuda"))
    q = (n, N, case["heads"], D)
    spread = 2.0 if case["cap"] else 1.0  # scores that the cap bends
    st["q"] = (torch.randn(q, generator=gen, device="cuda") * spread).to(dt)
    st["out"] = torch.empty(q, device="cuda", dtype=dt)
    st["lse"] = torch.empty(q[:3], device="cuda")
    st["slopes"] = None
    if case["slopes"]:
        h = torch.arange(1, case["heads"] + 1, dtype=torch.float64)
        st["slopes"] = torch.exp2(-8 * h / case["heads"]).float().cuda()
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    from ulysses_qkv_proj_gb300 import binding as qb
    case = st["case"]
    op = case["op"]
    if op == "table":
        qb.qnre_rope_table(st["out"], theta=st["theta"], first=st["first"], scaling=case["scaling"], factor=st["factor"],
                           original=st["original"])
        return st["out"]
    if op == "attention":
        qb.qnre_cache_shared_prefix(st["cache"], st["rows"], st["groups"], st["shared"])
        qb.qnre_prefix_attention(st["q"], st["cache"], 0, st["rows"], st["groups"], st["shared"], st["masks"], st["out"],
                                 lse=st["lse"], depths=st["depths"], softcap=case["cap"], slopes=st["slopes"],
                                 workspace=st["workspace"])
        return st["out"], st["lse"], st["shared"]
    settings = dict(temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
    if op == "sample":
        qb.qnre_sample(st["logits"], st["u"], st["tokens"], **settings)
        return st["tokens"]
    qb.qnre_filter_probs(st["logits"], st["probs"], **settings)
    return st["probs"]


# ------------------------------------------------------------------ the plain forms

def _frequencies(case, st):
    """Angle of one position for each pair of channels, and the factor on cos and sin."""
    rot, theta, s, original = case["rot"], st["theta"], st["factor"], st["original"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    kind = case["scaling"]
    if kind == "base":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if kind == "linear":
        f = f / s
    if kind == "yarn":  # by channel, between the ones that turn 32 times and once over the original length
        first, last = (rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32.0, 1.0))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
        ramp = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        return f * (ramp / s + 1 - ramp), 0.1 * math.log(s) + 1
    if kind == "wavelength":  # by the turns over the original length, from 1 to 4
        keep = ((original * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * (keep + (1 - keep) / s)
    return f, 1.0


def _table(st):
    case = st["case"]
    f, size = _frequencies(case, st)
    p = torch.arange(st["first"], st["first"] + case["n_pos"], dtype=torch.float64, device="cuda")
    a = p[:, None] * f
    return torch.cat([a.cos() * size, a.sin() * size], 1).float()


def _attention(st):
    case = st["case"]
    n, N, Hq, D = st["q"].shape
    Hk, page = case["kv_heads"], st["kpool"].shape[3]
    G = Hq // Hk
    out = torch.empty_like(st["q"])
    lse = torch.empty((n, N, Hq), device="cuda")
    bits = torch.arange(N, device="cuda")
    table = st["table"][st["rows"].long()]
    shared = []
    for a, b in zip(st["host_starts"], st["host_starts"][1:]):
        same = ((table[a:b] == table[a]) & (table[a] >= 0)).all(0).int().cumprod(0).sum()
        whole = st["lens"][st["rows"][a:b].long()].min() // page
        shared.append(torch.minimum(same, whole) * page * (b - a > 1))
    for i in range(n):
        L = st["host_lens"][i]
        blocks = _blocks(L + N, page)
        ids = table[i, :blocks].long()
        k = st["kpool"][0, ids].transpose(0, 1).reshape(Hk, blocks * page, D)[:, :L + N].float()
        v = st["vpool"][0, ids].transpose(0, 1).reshape(Hk, blocks * page, D)[:, :L + N].float()
        q = st["q"][i].float().view(N, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * N, D)
        s = (q @ k.transpose(1, 2)).view(Hk, G, N, L + N) * (1 / math.sqrt(D))
        if case["cap"]:
            s = torch.tanh(s / case["cap"]) * case["cap"]
        if case["slopes"]:
            depth = st["depths"][i]
            at = torch.cat([torch.arange(L, device="cuda"), L + depth])
            s = s + st["slopes"].view(Hk, G, 1, 1) * (at[None] - (L + depth)[:, None]).float()
        see = (st["masks"][i][:, None] >> bits[None]) & 1
        s[..., L:].masked_fill_(see == 0, float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        o = (p / z).view(Hk, G * N, L + N) @ v
        out[i] = o.view(Hk, G, N, D).permute(2, 0, 1, 3).reshape(N, Hq, D).to(out.dtype)
        lse[i] = (m + torch.log(z))[..., 0].permute(2, 0, 1).reshape(N, Hq)
    return out, lse, torch.stack(shared).int()


def _kept(x, T, k, p, m):
    """Weights [rows, V] in 64 bits, zero where the settings (a column each) leave a token out."""
    V = x.shape[-1]
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    z = order.values.double()
    w = torch.exp((z - z[:, :1]) / torch.where(T > 0, T.double(), 1.0))
    rank = torch.arange(V, device="cuda")[None]
    w = w * ((w >= m.double()) & ((k <= 0) | (rank < k)) & ((T > 0) | (rank < 1)))
    before = w.cumsum(-1) - w
    w = w * ((p >= 1) | (before < p.double() * w.sum(-1, keepdim=True)) | (rank == 0))
    return torch.empty_like(w).scatter_(1, order.indices, w)


def _sample(st):
    w = _kept(st["logits"], *(st[x][:, None] for x in ("temperature", "top_k", "top_p", "min_p")))
    c = w.cumsum(-1)
    pick = (c <= st["u"].double()[:, None] * c[:, -1:]).sum(-1)
    last = w.shape[1] - 1 - (w.flip(-1) > 0).int().argmax(-1)
    return torch.minimum(pick, last).int()


def _filter(st):
    n, N, V = st["logits"].shape
    out = torch.empty((n, N, V), device="cuda")
    for i in range(n):
        w = _kept(st["logits"][i], *(st[x][i].expand(N, 1) for x in ("temperature", "top_k", "top_p", "min_p")))
        out[i] = (w / w.sum(-1, keepdim=True)).float()
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"table": _table, "attention": _attention, "sample": _sample, "filter": _filter}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact results

def _exact_table(st):
    """One channel pair at a time on the host, each angle brought to (-pi, pi] before its cosine."""
    case = st["case"]
    rot, s, original = case["rot"], st["factor"], st["original"]
    out = torch.empty((case["n_pos"], rot), dtype=torch.float64)
    p = torch.arange(case["n_pos"], dtype=torch.float64) + st["first"]
    size = 1.0 + 0.1 * math.log(s) if case["scaling"] == "yarn" else 1.0
    base = st["theta"]
    if case["scaling"] == "base":
        base *= math.exp(math.log(s) * rot / (rot - 2))

    def channel(turns):  # the (fractional) pair that makes so many turns over the original length
        return math.log(original / (turns * 2 * math.pi)) / math.log(base) * rot / 2

    for i in range(rot // 2):
        f = math.exp(-math.log(base) * 2 * i / rot)
        if case["scaling"] == "linear":
            f /= s
        elif case["scaling"] == "yarn":
            lo, hi = max(math.floor(channel(32.0)), 0), min(math.ceil(channel(1.0)), rot - 1)
            slow = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = (1 - slow) * f + slow * f / s
        elif case["scaling"] == "wavelength":
            turns = original * f / (2 * math.pi)
            f = f if turns > 4 else f / s if turns < 1 else f / s + (f - f / s) * (turns - 1) / 3
        turn = torch.remainder(p * (f / (2 * math.pi)), 1.0)
        turn = torch.where(turn > 0.5, turn - 1, turn) * (2 * math.pi)
        out[:, i] = size * torch.cos(turn)
        out[:, rot // 2 + i] = size * torch.sin(turn)
    return out


def _exact_attention(st):
    case, page = st["case"], st["case"]["page"]
    n, N, Hq, D = st["q"].shape
    G = Hq // case["kv_heads"]
    out = torch.zeros((n, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, N, Hq), dtype=torch.float64, device="cuda")
    for i, L in enumerate(st["host_lens"]):
        at = torch.arange(L + N, device="cuda")
        pages = st["table"][st["host_rows"][i]].long()[at // page]
        node = torch.arange(N, device="cuda")
        hidden = torch.cat([torch.zeros((N, L), dtype=torch.bool, device="cuda"),
                            torch.bitwise_right_shift(st["masks"][i][:, None], node[None]) % 2 == 0], 1)
        place = at.double()
        place[L:] = L + st["depths"][i].double()
        for h in range(case["kv_heads"]):
            k = st["kpool"][0][pages, h, at % page].double()
            v = st["vpool"][0][pages, h, at % page].double()
            s = torch.einsum("tgd,ld->gtl", st["q"][i, :, h * G:(h + 1) * G].double(), k) / D ** 0.5
            if case["cap"]:
                e = torch.expm1(-2 * s.abs() / case["cap"])
                s = -torch.sign(s) * case["cap"] * e / (e + 2)
            if case["slopes"]:
                s = s - st["slopes"][h * G:(h + 1) * G].double()[:, None, None] * (place[L:, None] - place[None])
            s = torch.where(hidden[None], -math.inf, s)
            z = torch.logsumexp(s, -1)
            out[i, :, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", torch.exp(s - z[..., None]), v)
            lse[i, :, h * G:(h + 1) * G] = z.t()
    table, shared = st["table"].tolist(), []
    for a, b in zip(st["host_starts"], st["host_starts"][1:]):
        rows, blocks = st["host_rows"][a:b], 0
        while len(rows) > 1 and all((blocks + 1) * page <= st["host_lens"][i] and table[r][blocks] == table[rows[0]][blocks] >= 0
                                    for i, r in zip(range(a, b), rows)):
            blocks += 1
        shared.append(blocks * page)
    return out, lse, torch.tensor(shared, dtype=torch.int32)


def _exact_row(x, T, k, p, m):
    """The weights of one row's tokens, zero where left out: by the value of the last token that is kept."""
    x = x.double()
    if not T > 0:
        return torch.nn.functional.one_hot(x.argmax(), x.numel()).double()
    w = torch.exp((x - x.max()) / T)
    w[w < m] = 0
    if 0 < k < x.numel():
        least = torch.topk(x, k).values[-1]
        ties = (x == least).nonzero()[:, 0]
        gone = x < least
        gone[ties[k - int((x > least).sum()):]] = True
        w[gone] = 0
    if p < 1:
        room = p * w.sum()
        value, count = torch.unique(x[w > 0], return_counts=True)
        value, count = value.flip(0), count.flip(0)
        each = torch.exp((value - value[0]) / T)
        above = torch.cat([room.new_zeros(1), (each * count).cumsum(0)])
        g = int((above[:-1] < room).sum()) - 1          # the last value of which anything is kept
        g = max(g, 0)
        ties = ((x == value[g]) & (w > 0)).nonzero()[:, 0]
        stay = max(1 if g == 0 else 0, int(torch.ceil((room - above[g]) / each[g])))
        w[x < value[g]] = 0
        w[ties[stay:]] = 0
    return w


def _exact_rows(st, i, rows):
    args = [st[x][i].double().item() for x in ("temperature", "top_k", "top_p", "min_p")]
    return [_exact_row(r, args[0], int(args[1]), args[2], args[3]) for r in rows]


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "table":
        return _exact_table(st)
    if op == "attention":
        return _exact_attention(st)
    if op == "sample":
        out = []
        for i in range(case["n"]):
            w = _exact_rows(st, i, st["logits"][i:i + 1])[0]
            kept = w.nonzero()[:, 0]
            c = w[kept].cumsum(0)
            pick = int(torch.searchsorted(c, st["u"][i].double() * c[-1], right=True))
            out.append(int(kept[min(pick, len(kept) - 1)]))
        return torch.tensor(out, dtype=torch.int32)
    out = torch.empty(st["logits"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["n"]):
        for j, w in enumerate(_exact_rows(st, i, st["logits"][i])):
            out[i, j] = w / w.sum()
    return out
