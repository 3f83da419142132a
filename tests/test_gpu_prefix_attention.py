"""qnre_cache_shared_prefix against a walk over lists; qnre_prefix_attention against the 64-bit plain form.

Tolerance, element by element: half a step of the output type on the value; each weight p is rounded to the inputs' type before
the product (half a step of sum p |v|); the scores' fp32 products of D terms, scaled to base 2, and the exponential move each p
by at most (D + 16) 2^-24 |scale q.k| + 2^-20 relative, times sum p |v|, and lse by that.  A capped score is off by 2^-21 of the
cap more (1e-7 relative by the polynomials, 2^-22 of the cap by the exponentials), a distance bias by four roundings of it."""
import random

import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Groups of rows over common pages, in random pages and rows; unused slots NaN.  groups: (members, common tokens in whole
    pages); own: each request's tokens behind them; alone: requests outside every group, in front."""

    def __init__(self, groups, own, nodes=1, Hq=4, Hk=1, dim=128, page=16, dtype="bf16", alone=0, counts=None, seed=0, layers=2,
                 layer=1, cap=0.0, slopes=False, spread=1.0):
        dt = DT[dtype]
        self.rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
        self.nodes, self.layer, self.page, self.dt, self.cap, self.Hk = nodes, layer, page, dt, cap, Hk
        sizes = [s for s, _ in groups]
        self.starts = [alone + sum(sizes[:g]) for g in range(len(groups) + 1)]
        group = [-1] * alone + [g for g, s in enumerate(sizes) for _ in range(s)]
        n = self.n = len(group)
        own = [own[i % len(own)] for i in range(n)]
        self.common = [groups[g][1] // page * page if g >= 0 else 0 for g in group]
        self.lens = [c + o for c, o in zip(self.common, own)]
        self.counts = counts or [nodes] * n
        need = [-(-(L + c) // page) for L, c in zip(self.lens, self.counts)]
        pages = sum(need) + 4
        order = torch.randperm(pages, generator=gen).tolist()
        rows_total = n + 2
        self.rows = self.rng.sample(range(rows_total), n)
        self.table = torch.full((rows_total, max(need) + 2), -1, dtype=torch.int32)
        self.seq = torch.zeros(rows_total, dtype=torch.int32)
        nan = float("nan")
        self.k, self.v = (torch.full((layers, pages, Hk, page, dim), nan, dtype=dt) for _ in range(2))
        first = {}
        self.keys, self.values = [], []
        for i, r in enumerate(self.rows):
            shared = self.common[i] // page
            g = group[i]
            ids = [order.pop() for _ in range(need[i] - (shared if g in first else 0))]
            if g in first:
                ids = first[g][0] + ids
            self.table[r, :need[i]] = torch.tensor(ids, dtype=torch.int32)
            self.seq[r] = self.lens[i]
            T = self.lens[i] + self.counts[i]
            kk, vv = (torch.randn((T, Hk, dim), generator=gen).to(dt) for _ in range(2))
            if g in first:
                kk[:self.common[i]], vv[:self.common[i]] = first[g][1][:self.common[i]], first[g][2][:self.common[i]]
            elif g >= 0:
                first[g] = (ids[:shared], kk, vv)
            self.keys.append(kk)
            self.values.append(vv)
        self.fill()
        self.q = (torch.randn((n, nodes, Hq, dim), generator=gen) * spread).to(dt)
        self.parents = [D.random_tree(self.rng, nodes, 3) for _ in range(n)]
        self.masks = [D.ancestors(p)[0] for p in self.parents]
        self.depths = [D.ancestors(p)[1] for p in self.parents]
        self.scale = dim ** -0.5
        self.slopes = 2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq) if slopes else None

    def fill(self):
        for i, r in enumerate(self.rows):
            for x in range(len(self.keys[i])):
                at = (self.layer, int(self.table[r, x // self.page]), slice(None), x % self.page)
                self.k[at], self.v[at] = self.keys[i][x], self.values[i][x]

    def prepare(self, groups=True):
        qb = _qb()
        self.cache = qb.PagedCache(self.k.cuda(), self.v.cuda(), self.table.cuda(), self.seq.cuda(),
                                   torch.ones(self.k.shape[1], dtype=torch.int32, device="cuda"))
        self.d_rows, self.d_groups = _i32(self.rows), _i32(self.starts)
        self.d_shared = torch.full((len(self.starts) - 1,), -5, dtype=torch.int32, device="cuda")
        qb.qnre_cache_shared_prefix(self.cache, self.d_rows, self.d_groups, self.d_shared)
        q = self.q.cuda()
        self.out = torch.full(q.shape, 5.0, dtype=self.dt, device="cuda")
        self.lse = torch.full(q.shape[:3], 5.0, device="cuda")
        self.ws = qb.prefix_attention_workspace(q, self.cache, groups=groups)
        self.ws.fill_(255)
        return q

    def call(self, q, mask="tree", use_counts=False, groups=True, stream=None):
        n = self.n
        _qb().qnre_prefix_attention(
            q, self.cache, self.layer, self.d_rows, self.d_groups if groups else None, self.d_shared if groups else None,
            D.signed(self.masks).cuda() if mask == "tree" else None, self.out, lse=self.lse,
            counts=_i32(self.counts) if use_counts else None, depths=_i32(self.depths) if mask == "tree" and n else None,
            softcap=self.cap, slopes=None if self.slopes is None else self.slopes.cuda(), workspace=self.ws, stream=stream)

    def run(self, **kw):
        q = self.prepare(kw.get("groups", True))
        self.call(q, **kw)
        return self.out.cpu(), self.lse.cpu()

    def plain(self, i, chain=False):
        """out, lse and sum p |v| of request i, and the largest score before the cap and bias."""
        N, Hq, dim = self.q.shape[1:]
        L, c = self.lens[i], self.counts[i]
        G = Hq // self.Hk
        out, lse = torch.zeros(N, Hq, dim, dtype=torch.float64), torch.full((N, Hq), -torch.inf, dtype=torch.float64)
        size, bias_most = torch.zeros_like(out), 0.0
        for t in range(min(N, c)):
            see = list(range(L)) + [L + j for j in range(c) if (j <= t if chain else self.masks[i][t] >> j & 1)]
            if not see:
                continue
            k, v = self.keys[i][see].double(), self.values[i][see].double()
            depth = list(range(N)) if chain else self.depths[i]
            place = torch.tensor([x if x < L else L + depth[x - L] for x in see], dtype=torch.float64)
            for h in range(Hq):
                s = k[:, h // G] @ self.q[i, t, h].double() * self.scale
                if self.cap:
                    s = self.cap * torch.tanh(s / self.cap)
                if self.slopes is not None:
                    b = float(self.slopes[h]) * (place - (L + depth[t]))
                    bias_most = max(bias_most, float(b.abs().max()))
                    s = s + b
                lse[t, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[t, h])
                out[t, h] = p @ v[:, h // G]
                size[t, h] = p @ v[:, h // G].abs()
        return out, lse, size, bias_most

    def check(self, out, lse, status=0, chain=False, only=None):
        assert self.cache.status() == status
        half, dim = D.half_step(self.dt), self.q.shape[-1]
        for i in range(self.n) if only is None else only:
            ref, rl, size, bias = self.plain(i, chain)
            most = self.keys[i].double().norm(dim=-1).max() if len(self.keys[i]) else 0.0
            s = float(self.q[i].double().norm(dim=-1).max() * most * self.scale)
            rel = (dim + 16) * 2.0 ** -24 * s + 2.0 ** -20 + self.cap * 2.0 ** -21 + 4 * 2.0 ** -24 * bias
            tol = half * ref.abs() * 1.02 + (half + 2 * rel) * size + 1e-7
            err = (out[i].double() - ref).abs()
            assert not torch.isnan(err).any(), f"request {i}: NaN"
            assert (err <= tol).all(), f"request {i}: worst excess {(err - tol).max():.3g}"
            same = torch.isinf(rl)
            assert torch.equal(torch.isinf(lse[i]) & (lse[i] < 0), same)
            assert ((lse[i].double() - rl)[~same].abs() <= 2 * rel + 1e-6 * rl[~same].abs() + 1e-6).all()


def _walk(c):
    """Common tokens by a walk over each group's lists."""
    got = []
    table, seq = c.table.tolist(), c.seq.tolist()
    for a, b in zip(c.starts, c.starts[1:]):
        rows, blocks = c.rows[a:b], 0
        while len(rows) > 1 and all((blocks + 1) * c.page <= seq[r] and table[r][blocks] == table[rows[0]][blocks] >= 0 for r in rows):
            blocks += 1
        got.append(blocks * c.page)
    return got


SHAPES = [  # groups, own, keywords
    ([(1, 0)], [1], dict()),
    ([(2, 16)], [0], dict(nodes=1)),
    ([(5, 128), (1, 64), (3, 300)], [3, 0, 140], dict(Hq=8, Hk=2)),
    ([(9, 500)], [1, 129, 64], dict(Hq=8, Hk=1, dim=64, dtype="fp16", page=24)),
    ([(3, 200), (4, 130)], [17, 2], dict(nodes=5, Hq=4, Hk=2, alone=2)),
    ([(20, 260)], [5, 0, 90], dict(Hq=8, Hk=1)),                              # 160 rows: a cluster of two
    ([(40, 130), (3, 400), (9, 260)], [7, 30], dict(Hq=8, Hk=1, page=8)),     # a cluster's units and what they leave
    ([(6, 144)], [40, 1], dict(nodes=20, Hq=14, Hk=2, page=48)),              # 140 rows a request: units of nodes
    ([(2, 256), (2, 128)], [9], dict(nodes=64, Hq=8, Hk=1, dim=64, page=128)),
    ([(33, 512)], [200, 1, 30], dict(Hq=1, Hk=1, dim=64, page=256)),          # up to 128 requests a unit
    ([(7, 96)] * 5, [4, 250, 0], dict(Hq=7, Hk=1, dtype="fp16", page=32, alone=3)),
    ([(2, 1000)], [300, 5], dict(nodes=2, Hq=128, Hk=1, page=40)),            # 128 heads to one
]


@pytest.mark.parametrize("groups,own,kw", SHAPES)
def test_groups(groups, own, kw):
    c = Case(groups, own, seed=len(groups) + len(own), **kw)
    c.check(*c.run())
    assert c.d_shared.tolist() == _walk(c)


@pytest.mark.parametrize("groups,own,kw", [SHAPES[i] for i in (2, 4, 6, 7, 8)])
def test_rows_that_share_nothing(groups, own, kw):
    """Without groups: every row by itself, and what the tree attention gives."""
    c = Case(groups, own, seed=3, **kw)
    out, lse = c.run(groups=False)
    c.check(out, lse)
    qb = _qb()
    q, o2 = c.q.cuda(), torch.empty_like(c.out)
    qb.qnre_tree_attention(q, c.cache, c.layer, c.d_rows, D.signed(c.masks).cuda(), o2, workspace=qb.tree_attention_workspace(q, c.cache))
    c.check(o2.cpu(), lse)


@pytest.mark.parametrize("cap,slopes,spread", [(30.0, False, 1.0), (5.0, False, 4.0), (50.0, True, 8.0), (0.0, True, 1.0), (1e4, False, 1.0),
                                               (1e-6, False, 1.0)])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_caps_and_biases(cap, slopes, spread, dim, dtype):
    """Scores far below the cap, about it and beyond; positions by depth in the drafted trees."""
    c = Case([(5, 160), (12, 300)], [130, 2, 31], nodes=6, Hq=8, Hk=2, dim=dim, dtype=dtype, cap=cap, slopes=slopes, spread=spread, seed=5,
             alone=1)
    c.check(*c.run())


def test_bias_of_a_chain_and_rising_with_distance():
    c = Case([(4, 256)], [40, 3], nodes=7, Hq=4, Hk=2, slopes=True, seed=6)
    c.slopes = torch.tensor([0.5, -0.01, 0.0, -0.05])
    c.check(*c.run(mask=None), chain=True)


def test_many_requests_and_groups():
    """More than the short tables hold."""
    c = Case([(4, 32)] * 40 + [(1, 16)], [3, 0, 18], Hq=2, Hk=1, seed=7, alone=5)
    c.check(*c.run(), only=range(0, c.n, 7))
    c = Case([(300, 64)], [1, 20], Hq=2, Hk=2, dim=64, seed=8)
    c.check(*c.run(), only=range(0, 300, 23))


def test_counts_masks_and_empty_rows():
    """Requests with fewer nodes, rows without a token, nodes whose mask names nothing."""
    c = Case([(4, 32), (3, 0)], [0, 5, 0], nodes=6, Hq=4, Hk=2, counts=[6, 0, 3, 1, 0, 6, 2], seed=9)
    c.check(*c.run(use_counts=True))
    c = Case([(3, 0)], [0], nodes=4, Hq=2, Hk=1, seed=10)
    c.masks = [[0, 1, 0, 15]] * 3
    c.check(*c.run())


def test_shared_may_be_smaller_or_larger():
    """Any whole number of pages that is common serves; more than a member has is cut off; groups that overlap or descend
    are read as ascending."""
    c = Case([(4, 320), (3, 160)], [40, 7], Hq=4, Hk=2, seed=11)
    q = c.prepare()
    for shared in ([320, 160], [64, 0], [16, 160], [-3, 7], [320, 96]):
        c.d_shared.copy_(torch.tensor(shared))
        c.out.fill_(3), c.ws.fill_(255)
        c.call(q)
        c.check(c.out.cpu(), c.lse.cpu())
    short = c.rows[2]  # a member that was cut back
    c.seq[short] = c.lens[2] = 50
    c.keys[2], c.values[2] = torch.cat([c.keys[2][:50], c.keys[2][50:51]]), torch.cat([c.values[2][:50], c.values[2][50:51]])
    c.cache.seq_lens.copy_(c.seq)
    c.d_shared.copy_(torch.tensor([320, 160]))
    c.call(q)
    c.check(c.out.cpu(), c.lse.cpu())
    c.d_groups.copy_(torch.tensor([7, 4, 2]))
    c.call(q)
    c.check(c.out.cpu(), c.lse.cpu())


def test_a_row_twice_and_rows_outside():
    c = Case([(3, 96)], [20], Hq=4, Hk=2, seed=12)
    q = c.prepare()
    c.d_rows = _i32([c.rows[0], 1000, -1])
    c.call(q, groups=False)
    out = c.out.cpu()
    c.check(out, c.lse.cpu(), status=0x2, only=[0])
    assert not out[1:].any() and torch.isinf(c.lse[1:]).all()
    c.call(q)                                        # a group with such rows shares nothing
    c.check(c.out.cpu(), c.lse.cpu(), status=0x2, only=[0])
    c.d_rows = _i32([c.rows[0]] * 3)                 # three samples of one row
    _qb().qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
    assert c.d_shared.tolist() == [c.lens[0] // 16 * 16]
    c.call(q)
    for i in (1, 2):
        c.keys[i], c.values[i], c.lens[i], c.masks[i] = c.keys[0], c.values[0], c.lens[0], c.masks[0]
    c.check(c.out.cpu(), c.lse.cpu())


def test_missing_pages_are_zeros():
    c = Case([(3, 96)], [40], Hq=4, Hk=2, seed=13)
    q = c.prepare()
    r = c.rows[1]
    c.cache.block_table[r, 7] = -1                   # in a row's own tokens
    c.keys[1][112:128] = 0
    c.values[1][112:128] = 0
    c.call(q)
    c.check(c.out.cpu(), c.lse.cpu(), status=0x4)
    for r in c.rows:
        c.cache.block_table[r, 2] = c.k.shape[1] + 3  # in the common ones, a page beyond the cache
    for i in range(3):
        c.keys[i][32:48] = 0
        c.values[i][32:48] = 0
    c.call(q)
    c.check(c.out.cpu(), c.lse.cpu(), status=0x4)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("where", ["common", "own"])
def test_infinite_values_reach_their_rows_alone(dtype, dim, where):
    """An infinite V gives infinity (NaN for both signs) in the rows that see it, whatever its weight, and nothing elsewhere,
    although rows of other requests lie in the same product."""
    c = Case([(6, 300), (7, 160)], [50, 200, 3], nodes=2, Hq=4, Hk=2, dim=dim, dtype=dtype, seed=14)
    i, x = 2, 100 if where == "common" else c.common[2] + 1
    hit = [j for j in range(c.n) if (0 <= j < 6 if where == "common" else j == i)]
    inf = float("inf")
    for j in hit:
        c.values[j][x, 0, 3], c.values[j][x, 0, 5] = inf, -inf
        c.values[j][x - 1, 0, 5] = inf
        c.values[j][x, 1, 8] = float("nan")
        c.keys[j][x] = -4.0 * c.q[i, 0, 0].sign() * c.q[i, 0, 0].abs().clamp(min=0.5)   # with hardly any weight for some
    c.fill()
    out, lse = c.run()
    for j in hit:
        assert (out[j, :, :2, 3] == inf).all() and torch.isnan(out[j, :, :2, 5]).all() and torch.isnan(out[j, :, 2:, 8]).all()
        out[j, :, :2, 3] = out[j, :, :2, 5] = out[j, :, 2:, 8] = 0
    for j in hit:
        c.values[j][x, 0, 3] = c.values[j][x, 0, 5] = c.values[j][x - 1, 0, 5] = c.values[j][x, 1, 8] = 0
    sane = torch.ones(c.q.shape[2:], dtype=torch.bool)
    sane[:2, 3] = sane[:2, 5] = sane[2:, 8] = False
    whole = c.plain
    c.plain = lambda k, chain=False: (lambda r: (r[0] * sane if k in hit else r[0], *r[1:]))(whole(k, chain))
    c.check(out, lse)


def test_strange_keys_stay_with_their_request():
    c = Case([(9, 64)], [30, 4], nodes=2, Hq=4, Hk=2, seed=15)
    c.keys[4][c.common[4] + 2, 0] = float("nan")
    c.keys[7][c.common[7], 1] = float("inf")
    c.fill()
    out, lse = c.run()
    assert torch.isnan(out[4, :, :2]).all()
    c.check(out, lse, only=[0, 1, 2, 3, 5, 6, 8])


def test_drafts_that_others_do_not_see():
    """Non-finite K and V of a drafted node reach only the nodes whose mask names it, and no other request."""
    c = Case([(5, 48)], [10, 3], nodes=8, Hq=4, Hk=2, dim=64, seed=16)
    L = c.lens[1]
    c.values[1][L + 3, 0, 7] = float("inf")
    c.values[1][L + 5] = float("nan")
    c.masks[1] = [(1 << (t + 1)) - 1 & ~0b101000 | 1 << t for t in range(8)]
    c.fill()
    out, lse = c.run()
    assert torch.isnan(out[1, 5]).all() and (out[1, 3, :2, 7] == float("inf")).all()
    clean = c.values[1].clone()
    c.values[1] = torch.where(torch.isfinite(clean), clean, torch.zeros_like(clean))
    out[1, 5] = 0
    out[1, 3, :2, 7] = 0
    ref = c.plain(1)
    tol = D.half_step(c.dt) * (ref[0].abs() + ref[2]) * 1.1 + 1e-3
    keep = torch.ones_like(ref[0], dtype=torch.bool)
    keep[5] = False
    keep[3, :2, 7] = False
    assert ((out[1].double() - ref[0]).abs() <= tol)[keep].all()
    c.check(out, lse, only=[0, 2, 3, 4])


def test_queries_as_views():
    """q as a slice of a token-major projection and by heads; the same bits as a copy."""
    c = Case([(4, 160)], [33, 2], nodes=3, Hq=8, Hk=2, seed=17)
    q = c.prepare()
    c.call(q)
    want = c.out.clone()
    wide = torch.zeros((c.n, 3, 12, 128), dtype=c.dt, device="cuda")
    wide[:, :, 2:10] = q
    heads = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    for view in (wide[:, :, 2:10], heads):
        c.out.fill_(1)
        c.call(view)
        assert torch.equal(c.out, want)


def test_replays_follow_the_lengths():
    """Captured with the search for common tokens; lengths, tables and groups change between replays; same bits as call by call."""
    qb = _qb()
    c = Case([(6, 320), (5, 160)], [90, 4, 200], Hq=8, Hk=2, seed=18)
    q = c.prepare()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        masks = D.signed(c.masks).cuda()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qb.qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
            qb.qnre_prefix_attention(q, c.cache, c.layer, c.d_rows, c.d_groups, c.d_shared, masks, c.out, lse=c.lse, workspace=c.ws)
    for step in range(3):
        if step == 1:
            c.d_groups.copy_(torch.tensor([0, 3, 11]))
        if step == 2:
            c.cache.seq_lens[c.rows[1]] = 70
            c.lens[1] = 70
            c.keys[1], c.values[1] = c.keys[1][:71], c.values[1][:71]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        got = c.out.clone(), c.lse.clone()
        qb.qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
        c.call(q)
        assert torch.equal(c.out, got[0]) and torch.equal(c.lse, got[1])
        c.check(got[0].cpu(), got[1].cpu())


def test_two_streams_with_a_workspace_each():
    cases = [Case([(8, 480)], [90, 4], Hq=8, Hk=2, seed=19), Case([(30, 96)], [5, 40], Hq=4, Hk=1, dim=64, dtype="fp16", seed=20)]
    qs = [c.prepare() for c in cases]
    want = []
    for c, q in zip(cases, qs):
        c.call(q)
        want.append(c.out.clone())
        c.out.fill_(0)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, q, s in zip(cases, qs, streams):
            c.call(q, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.out, w) for c, w in zip(cases, want))


def test_without_lse_and_with_another_scale():
    qb = _qb()
    c = Case([(3, 64)], [9], Hq=4, Hk=2, seed=21)
    q = c.prepare()
    c.scale = 0.2
    qb.qnre_prefix_attention(q, c.cache, c.layer, c.d_rows, c.d_groups, c.d_shared, D.signed(c.masks).cuda(), c.out, scale=0.2, workspace=c.ws)
    assert (c.lse == 5).all()
    lse = torch.stack([c.plain(i)[1] for i in range(c.n)]).float()
    c.check(c.out.cpu(), lse)
    qb.qnre_prefix_attention(q[:0], c.cache, c.layer, c.d_rows[:0], None, None, None, c.out[:0], workspace=c.ws)


@pytest.mark.parametrize("blocks", [1, 31, 256, 257, 700])
@pytest.mark.parametrize("n", [2, 37, 400])
def test_common_pages(blocks, n):
    """Random tables that part at random places; missing and foreign pages end what is common."""
    qb = _qb()
    rng = random.Random(blocks * n)
    ps = 16
    pages = blocks + n + 5
    table = torch.full((n, blocks + 2), -1, dtype=torch.int32)
    seq = []
    starts, at = [0], 0
    while at < n:
        at = min(n, at + rng.choice([1, 2, 3, 50]))
        starts.append(at)
    for a, b in zip(starts, starts[1:]):
        base = [rng.randrange(blocks) for _ in range(blocks)]
        part = rng.randint(0, blocks)
        for i in range(a, b):
            ids = list(base)
            if rng.random() < 0.5 and part < blocks:
                ids[part] = blocks + i
            if rng.random() < 0.1:
                ids[rng.randrange(blocks)] = rng.choice([-1, pages + 2])
            table[i, :blocks] = torch.tensor(ids, dtype=torch.int32)
            seq.append(rng.choice([blocks * ps, blocks * ps - rng.randint(0, blocks * ps - 1), blocks * ps - 1]))
    pool = torch.zeros((1, pages, 1, ps, 64), dtype=torch.bfloat16, device="cuda")
    cache = qb.PagedCache(pool, torch.zeros_like(pool), table.cuda(), _i32(seq), torch.ones(pages, dtype=torch.int32, device="cuda"))
    want = []
    for a, b in zip(starts, starts[1:]):
        k = 0
        while b - a > 1 and k < blocks and all((k + 1) * ps <= seq[i] and table[i, k] == table[a, k] and 0 <= table[a, k] < pages
                                               for i in range(a, b)):
            k += 1
        want.append(k * ps)
    order = list(range(n))
    shared = torch.full((len(starts) - 1,), -1, dtype=torch.int32, device="cuda")
    qb.qnre_cache_shared_prefix(cache, _i32(order), _i32(starts), shared)
    assert shared.tolist() == want and cache.status() == 0


def test_common_pages_of_rows_outside_the_cache():
    qb = _qb()
    c = Case([(3, 64), (2, 32)], [5], seed=22)
    c.prepare()
    c.d_rows[1] = 99
    qb.qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
    assert c.d_shared.tolist() == [0, 32] and c.cache.status() == 0x2
    c.d_groups.copy_(torch.tensor([3, 5, 4]))      # an empty one behind it
    qb.qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
    assert c.d_shared.tolist() == [32, 0] and c.cache.status() == 0
