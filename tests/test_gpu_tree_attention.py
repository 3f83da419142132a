"""qnre_tree_attention against the 64-bit plain form.

Tolerance, element by element: half a step of the output type on the value; each
weight p is rounded to the inputs' type before the product (half a step of sum p |v|);
the scores' fp32 products of D terms, scaled to base 2, and the exponential move each p by
at most (D + 16) 2^-24 |scale q.k| + 2^-20 relative, times sum p |v|, and lse by that."""
import random

import numpy as np
import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


class Case:
    """A cache with random pages in random order, every unused slot NaN, and q for drafted trees."""

    def __init__(self, lens, nodes, Hq, Hk, dim, page, dtype, branch=3, layers=2, layer=1, seed=0, counts=None):
        qb, dt = _qb(), DT[dtype]
        self.rng = random.Random(seed)
        gen = torch.Generator().manual_seed(seed)
        n = len(lens)
        self.lens, self.nodes, self.layer, self.page, self.dt = lens, nodes, layer, page, dt
        self.counts = counts or [nodes] * n
        need = [-(-(L + c) // page) for L, c in zip(lens, self.counts)]
        blocks, rows_total = max(need) + 1, n + 2
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen).tolist()
        self.table = torch.full((rows_total, blocks), -1, dtype=torch.int32)
        self.rows = self.rng.sample(range(rows_total), n)
        seq = torch.zeros(rows_total, dtype=torch.int32)
        nan = float("nan")
        self.k, self.v = (torch.full((layers, pages, Hk, page, dim), nan, dtype=dt) for _ in range(2))
        self.keys, self.values = [], []
        at = 0
        for i, r in enumerate(self.rows):
            ids = order[at:at + need[i]]
            at += need[i]
            self.table[r, :need[i]] = torch.tensor(ids, dtype=torch.int32)
            seq[r] = lens[i]
            T = lens[i] + self.counts[i]
            kk, vv = (torch.randn((T, Hk, dim), generator=gen).to(dt) for _ in range(2))
            self.keys.append(kk)
            self.values.append(vv)
            for x in range(T):
                self.k[layer, ids[x // page], :, x % page] = kk[x]
                self.v[layer, ids[x // page], :, x % page] = vv[x]
        self.seq = seq
        self.q = torch.randn((n, nodes, Hq, dim), generator=gen).to(dt)
        self.parents = [D.random_tree(self.rng, nodes, branch) for _ in lens]
        self.masks = [D.ancestors(p)[0] for p in self.parents]
        self.scale = dim ** -0.5

    def visible(self, i):
        L, c = self.lens[i], self.counts[i]
        vis = torch.zeros((self.nodes, L + c), dtype=torch.bool)
        for t in range(min(c, self.nodes)):
            vis[t, :L] = True
            for j in range(c):
                vis[t, L + j] = bool(self.masks[i][t] >> j & 1)
        return vis

    def run(self, mask="tree", use_counts=False, q=None):
        qb = _qb()
        pages = self.k.shape[1]
        self.cache = qb.PagedCache(self.k.cuda(), self.v.cuda(), self.table.cuda(), self.seq.cuda(),
                                   torch.ones(pages, dtype=torch.int32, device="cuda"))
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, 5.0, dtype=self.dt, device="cuda")
        lse = torch.full(q.shape[:3], 5.0, device="cuda")
        ws = qb.tree_attention_workspace(q, self.cache)
        ws.fill_(255)
        masks = D.signed(self.masks).cuda() if mask == "tree" else None
        counts = torch.tensor(self.counts, dtype=torch.int32).cuda() if use_counts else None
        rows = torch.tensor(self.rows, dtype=torch.int32).cuda()
        qb.qnre_tree_attention(q, self.cache, self.layer, rows, masks, out, lse=lse, counts=counts, workspace=ws)
        return out.cpu(), lse.cpu()

    def check(self, out, lse, status=0):
        assert self.cache.status() == status
        half, dim = D.half_step(self.dt), self.q.shape[-1]
        for i in range(len(self.lens)):
            ref, rl, size = D.attention(self.q[i], self.keys[i], self.values[i], self.visible(i), self.scale)
            s = (self.q[i].double().norm(dim=-1).max() * (self.keys[i].double().norm(dim=-1).max() if len(self.keys[i])
                                                           else 0.0) * self.scale)
            rel = float((dim + 16) * 2.0 ** -24 * s + 2.0 ** -20)
            tol = half * ref.abs() * 1.02 + (half + 2 * rel) * size + 1e-7
            err = (out[i].double() - ref).abs()
            assert not torch.isnan(err).any(), f"request {i}: NaN"
            assert (err <= tol).all(), f"request {i}: worst excess {(err - tol).max():.3g}"
            same = torch.isinf(rl)
            assert torch.equal(torch.isinf(lse[i]) & (lse[i] < 0), same)
            assert ((lse[i].double() - rl)[~same].abs() <= 2 * rel + 1e-6 * rl[~same].abs() + 1e-6).all()


SHAPES = [  # lens, nodes, Hq, Hk, dim, page, dtype
    ([1], 1, 1, 1, 128, 16, "bf16"),
    ([0], 1, 4, 4, 64, 8, "fp16"),                      # no context at all
    ([127, 128, 129, 0, 255], 1, 8, 2, 128, 16, "bf16"),
    ([300, 5, 1000], 3, 6, 1, 64, 24, "bf16"),          # pages that end inside a tile, group of 6
    ([700], 1, 32, 8, 128, 128, "fp16"),
    ([40, 513], 9, 8, 2, 128, 64, "bf16"),              # 36 rows: two copies
    ([90, 200, 3], 16, 7, 1, 128, 48, "fp16"),          # 112 rows: one copy
    ([260, 77], 33, 8, 1, 64, 32, "bf16"),              # 264 rows: three row tiles
    ([65, 1], 64, 4, 2, 128, 16, "bf16"),               # 64 nodes, drafts across a tile's edge
    ([5000, 1], 2, 4, 2, 128, 256, "bf16"),
    ([11, 130, 64, 64, 200, 1, 0, 90], 61, 3, 3, 64, 16, "fp16"),
]


@pytest.mark.parametrize("lens,nodes,Hq,Hk,dim,page,dtype", SHAPES)
def test_trees(lens, nodes, Hq, Hk, dim, page, dtype):
    c = Case(lens, nodes, Hq, Hk, dim, page, dtype, seed=len(lens) + nodes)
    c.check(*c.run())


@pytest.mark.parametrize("lens,nodes,Hq,Hk,dim,page,dtype", [
    ([300, 0, 77], 20, 14, 2, 128, 16, "bf16"),         # 18 nodes a tile: two row tiles share K and V
    ([200, 1000], 64, 8, 1, 64, 128, "fp16"),           # four
    ([90, 129], 40, 16, 1, 128, 8, "bf16"),             # five: two groups, the second with three idle CTAs
    ([500], 64, 32, 2, 128, 24, "bf16"),                # eight
    ([260], 2, 128, 1, 128, 64, "fp16"),                # 128 heads to one
])
def test_row_tiles_that_share_tokens(lens, nodes, Hq, Hk, dim, page, dtype):
    c = Case(lens, nodes, Hq, Hk, dim, page, dtype, seed=nodes + Hq)
    c.check(*c.run())


def test_queries_laid_out_by_heads():
    c = Case([150, 3], 5, 8, 2, 128, 16, "bf16", seed=13)
    q = c.q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    c.check(*c.run(q=q))


@pytest.mark.parametrize("nodes,G", [(1, 4), (5, 8), (40, 8)])
def test_long_context_spread_over_the_machine(nodes, G):
    c = Case([20011], nodes, 2 * G, 2, 128, 64, "bf16", seed=9)
    c.check(*c.run())


def test_chain_mask_and_ragged_counts():
    c = Case([50, 0, 300, 128], 7, 8, 2, 128, 16, "bf16", seed=4, counts=[7, 3, 0, 1])
    c.masks = [[(1 << (t + 1)) - 1 for t in range(7)] for _ in range(4)]
    out, lse = c.run(mask=None, use_counts=True)
    c.check(out, lse)
    assert not out[2].any() and not out[0, 7:].any() and torch.isinf(lse[2]).all()


def test_masks_that_leave_a_row_empty_or_see_single_nodes():
    c = Case([0, 0, 10], 5, 4, 2, 64, 8, "fp16", seed=5)
    c.masks = [[0, 1 << 3, 0, 0b11111, 1 << 4], [0] * 5, [0, 0, 1, 0, -1 & ((1 << 64) - 1)]]
    out, lse = c.run()
    c.check(out, lse)
    assert not out[1].any() and (lse[1] == float("-inf")).all()


def test_what_is_not_seen_never_arrives():
    """NaN and infinities in drafted slots that only some nodes see."""
    c = Case([120], 12, 8, 2, 128, 16, "bf16", seed=6)
    c.masks = [[1 << t for t in range(12)]]
    clean = c.run()
    c.check(*clean)
    for x, val in ((124, float("nan")), (130, float("inf")), (131, float("-inf"))):
        page, slot = c.table[c.rows[0], x // 16], x % 16
        c.k[1, page, :, slot, 3] = float("nan") if x == 124 else 0.0
        c.v[1, page, :, slot, 7] = val
    out, lse = c.run()
    keep = [t for t in range(12) if t not in (4, 10, 11)]
    # the other nodes' keys changed nowhere but in slots they do not see
    assert torch.equal(out[0, keep], clean[0][0, keep]) and torch.equal(lse[0, keep], clean[1][0, keep])
    assert torch.isnan(out[0, 4]).all()                       # its own key is NaN
    assert torch.isinf(out[0, 10, :, 7]).all() and (out[0, 10, :, 7] > 0).all()
    assert torch.isinf(out[0, 11, :, 7]).all() and (out[0, 11, :, 7] < 0).all()
    cols = [i for i in range(128) if i != 7]
    assert torch.isfinite(out[0, 10][:, cols]).all() and torch.isfinite(out[0, 11][:, cols]).all()


def test_what_is_not_seen_never_arrives_in_a_pair_of_row_tiles():
    """The same where two row tiles share K and V, in both halves of V's channels."""
    c = Case([120, 300], 40, 16, 2, 128, 16, "bf16", seed=14)
    c.masks = [[1 << t for t in range(40)] for _ in range(2)]
    clean = c.run()
    c.check(*clean)
    for i, L in enumerate(c.lens):
        for t, col in ((5, 3), (39, 90)):
            page, slot = c.table[c.rows[i], (L + t) // 16], (L + t) % 16
            c.v[1, page, :, slot, col] = float("inf")
    out, lse = c.run()
    keep = [t for t in range(40) if t not in (5, 39)]
    assert torch.equal(out[:, keep], clean[0][:, keep]) and torch.equal(lse, clean[1])
    for t, col in ((5, 3), (39, 90)):
        assert torch.isinf(out[:, t, :, col]).all()
        cols = [x for x in range(128) if x != col]
        assert torch.isfinite(out[:, t][..., cols]).all()


def test_large_scores_and_rising_maxima():
    """Scores far apart, rising along the context: the running maximum moves many times."""
    c = Case([900], 2, 4, 2, 64, 16, "fp16", seed=7)
    with torch.no_grad():
        ramp = torch.linspace(0.1, 6.0, 902)[:, None, None]
        c.keys[0] = (c.q[0, 0, :2].float()[None] * ramp * 0.5).to(c.dt)
        for x in range(902):
            c.k[1, c.table[c.rows[0], x // 16], :, x % 16] = c.keys[0][x]
    c.check(*c.run())


def test_strided_queries_and_repeatability():
    c = Case([333, 20, 1500], 6, 8, 2, 128, 32, "bf16", seed=8)
    buf = torch.zeros((6, 3, 12, 128), dtype=torch.bfloat16, device="cuda")
    view = buf.transpose(0, 1)[:, :, 2:10]
    view.copy_(c.q)
    a = c.run(q=view)
    c.check(*a)
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_requests():
    rng = random.Random(3)
    c = Case([rng.randint(0, 60) for _ in range(300)], 1, 2, 1, 64, 8, "bf16", seed=10)
    c.check(*c.run())


def test_bad_tables_are_reported():
    """A missing page reads as zeros, a bad row sees nothing; the other requests keep their results."""
    qb = _qb()
    c = Case([100, 40], 2, 4, 2, 128, 16, "bf16", seed=11)
    c.table[c.rows[1], 1] = 10 ** 6
    out, lse = c.run()
    assert c.cache.status() == qb.CACHE_BAD_PAGE
    c.keys[1][16:32] = 0
    c.values[1][16:32] = 0
    c.check(out, lse)
    c.rows = [c.rows[0], 99]
    out, lse = c.run()
    assert c.cache.status() == qb.CACHE_BAD_ROW and not out[1].any() and torch.isinf(lse[1]).all()


def test_graph_replay_on_grown_rows():
    """A captured call follows the cache's lengths and contents."""
    qb = _qb()
    c = Case([70, 10], 3, 8, 2, 128, 16, "bf16", seed=12)
    c.run()
    q, cache = c.q.cuda(), c.cache
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = qb.tree_attention_workspace(q, cache)
    rows, masks = torch.tensor(c.rows, dtype=torch.int32).cuda(), D.signed(c.masks).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qb.qnre_tree_attention(q, cache, 1, rows, masks, out, lse=lse, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    c.check(out.cpu(), lse.cpu())
    c.lens = [66, 7]
    cache.seq_lens[rows.long()] = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    g.replay()
    torch.cuda.synchronize()
    c.keys = [k[:L + 3] for k, L in zip(c.keys, c.lens)]
    c.values = [v[:L + 3] for v, L in zip(c.values, c.lens)]
    c.check(out.cpu(), lse.cpu())


@pytest.mark.parametrize("lens,nodes,Hq,Hk,dtype", [
    ([1000, 700, 1300, 128, 129, 1, 900, 1100], 2, 28, 14, "bf16"),  # runs of several tiles that span units, one tile alone
    ([1500, 1023, 900, 255, 1, 640], 20, 28, 14, "fp16"),
    ([384, 2, 1400, 900], 40, 14, 14, "fp16"),
])
def test_narrow_heads_over_runs_of_tiles(lens, nodes, Hq, Hk, dtype):
    """D = 64, scores rising along the context; then a draft's infinite values, seen by itself alone."""
    c = Case(lens, nodes, Hq, Hk, 64, 16, dtype, seed=21)
    for i, L in enumerate(lens):
        T = L + nodes
        ramp = torch.linspace(-2.0, 5.0, T)[:, None, None]
        c.keys[i] = (c.q[i, 0, ::Hq // Hk].float()[None] * ramp * 0.4).to(c.dt)
        for x in range(T):
            c.k[1, c.table[c.rows[i], x // 16], :, x % 16] = c.keys[i][x]
    c.masks = [[1 << t for t in range(nodes)] for _ in lens]
    clean = c.run()
    c.check(*clean)
    for i, L in enumerate(lens):
        x = L + nodes - 1
        c.v[1, c.table[c.rows[i], x // 16], :, x % 16, 33] = float("inf")
    out, lse = c.run()
    assert torch.equal(out[:, :-1], clean[0][:, :-1]) and torch.equal(lse, clean[1])
    assert torch.isinf(out[:, -1, :, 33]).all()
    cols = [x for x in range(64) if x != 33]
    assert torch.equal(out[:, -1][..., cols], clean[0][:, -1][..., cols])


def test_pools_and_tensors_outside_this_gpu_are_refused():
    """Pools in the host's memory, at the C entry itself (with one row tile and with several); then tensors of the CPU."""
    import ctypes
    qb = _qb()
    lib = qb.load_library()
    c = Case([20, 3], 20, 16, 2, 128, 16, "bf16", seed=2)
    for nodes in (1, 20):
        q = c.q[:, :nodes].contiguous().cuda()
        c.run()
        ws = qb.tree_attention_workspace(q, c.cache)
        rows = torch.tensor(c.rows, dtype=torch.int32).cuda()
        out = torch.full_like(q, 5.0)
        pinned = [t.pin_memory() for t in (c.k, c.v)]
        for which in range(2):
            s = qb._Cache.from_buffer_copy(c.cache._struct)
            setattr(s, "kv"[which], pinned[which].data_ptr())
            st = lib.qnre_tree_attention(qb._view4(q), ctypes.byref(s), c.layer, rows.data_ptr(), None, None, c.scale,
                                         out.data_ptr(), None, ws.data_ptr(), ws.numel(), qb._stream_ptr(None))
            assert st == 1
        with pytest.raises(qb.QnreError):
            qb.qnre_tree_attention(q, c.cache, c.layer, rows.cpu(), None, out, workspace=ws)
        with pytest.raises(qb.QnreError):
            qb.qnre_tree_attention(q, c.cache, c.layer, rows, None, out.cpu(), workspace=ws)
        torch.cuda.synchronize()
        assert (out == 5.0).all()
    cpu = qb.PagedCache(c.k, c.v, c.table, c.seq, torch.ones(c.k.shape[1], dtype=torch.int32))
    with pytest.raises(qb.QnreError):
        qb.qnre_cache_truncate(cpu, rows.cpu(), rows.cpu())


def _place(c, i, x, col, val):
    """Element `col` of V of token x of request i, in every head."""
    c.v[c.layer, c.table[c.rows[i], x // c.page], :, x % c.page, col] = val
    c.values[i][x, :, col] = val


SEEN = [  # lens, nodes, Hq, Hk, dim, page, dtype: rows laid out four times, twice, once, and shared by row tiles
    ([300, 5, 1000], 1, 8, 2, 128, 16, "bf16"),
    ([300, 5, 1000], 1, 8, 2, 64, 24, "fp16"),
    ([257, 128, 700], 5, 16, 2, 128, 16, "fp16"),
    ([257, 128, 700], 5, 16, 2, 64, 16, "bf16"),
    ([300, 130, 1000], 16, 14, 2, 128, 32, "bf16"),
    ([300, 130, 1000], 16, 14, 2, 64, 32, "fp16"),
    ([300, 130], 40, 16, 2, 128, 16, "bf16"),
    ([300, 130], 64, 8, 2, 64, 16, "fp16"),
    ([40000], 1, 8, 2, 128, 64, "bf16"),            # units that span many CTAs
    ([40000], 20, 16, 2, 64, 64, "fp16"),
]


@pytest.mark.parametrize("lens,nodes,Hq,Hk,dim,page,dtype", SEEN)
def test_infinite_values_in_the_context(lens, nodes, Hq, Hk, dim, page, dtype):
    """+inf, -inf, both, and NaN in V of cached tokens, first, last and between; one request stays finite."""
    c = Case(lens, nodes, Hq, Hk, dim, page, dtype, seed=nodes + dim)
    finite = [v.clone() for v in c.values]
    inf = float("inf")
    for i, L in enumerate(lens):
        if i == 1:
            continue
        for x, col, val in ((0, 3, inf), (L - 1, 20, -inf), (L // 2, 33, inf), (1, 33, -inf), (L // 3, dim - 1, float("nan")),
                            (L - 1, dim - 2, inf), (2, dim - 2, inf)):
            _place(c, i, x, col, val)
    out, lse = c.run()
    special, want = [3, 20, 33, dim - 1, dim - 2], torch.tensor([inf, -inf, float("nan"), float("nan"), inf])
    for i in range(len(lens)):
        if i != 1:
            got = out[i][..., special].float()
            assert torch.equal(torch.isnan(got), torch.isnan(want).expand_as(got))
            assert torch.equal(got.nan_to_num(0.0, inf, -inf), want.nan_to_num(0.0, inf, -inf).expand_as(got))
            out[i][..., special] = 0
            finite[i][..., special] = 0
    c.values = finite
    c.check(out, lse)


@pytest.mark.parametrize("nodes,Hq", [(1, 8), (5, 16), (16, 14)])
@pytest.mark.parametrize("dtype,below", [("bf16", 40.0), ("fp16", 25.0)])
def test_infinite_values_of_hardly_any_weight(nodes, Hq, dtype, below):
    """The infinite token's score lies far below another's: its weight counts, however few bits it is rounded to."""
    c = Case([200], nodes, Hq, 2, 128, 16, dtype, seed=3)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    for x in range(200 + nodes):
        c.keys[0][x] = 0
        c.keys[0][x, :, 0] = 0.0 if x else below / (8.0 * c.scale)
        c.k[1, c.table[c.rows[0], x // 16], :, x % 16] = c.keys[0][x]
    c.masks = [[(1 << 64) - 1 >> 64 - nodes] * nodes]
    _place(c, 0, 77, 5, float("inf"))
    _place(c, 0, 78, 100, float("-inf"))
    out, lse = c.run()
    assert (out[0, ..., 5] == float("inf")).all() and (out[0, ..., 100] == float("-inf")).all()
    for x, col in ((77, 5), (78, 100)):
        c.values[0][x, :, col] = 0
    out[0, ..., 5] = out[0, ..., 100] = 0
    c.values[0][:, :, [5, 100]] = 0
    c.check(out, lse)


@pytest.mark.parametrize("nodes", [1, 10, 20])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_small_weights_under_a_large_one(nodes, dtype):
    """10^5 tokens 17.5 nats under one score keep their share.  On top of the roundings above, fp16 weights below
    2^-21 of the largest are off by up to 2^-32 of it each.  As many requests of the same row as there are
    multiprocessors, so that a row's tokens are not divided."""
    T, n = 100000, torch.cuda.get_device_properties(0).multi_processor_count
    c = Case([T - nodes], nodes, 4, 1, 64, 64, dtype, seed=nodes)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    c.keys[0][:] = 0
    c.keys[0][7, :, 0] = 17.5 / (8.0 * c.scale)
    c.values[0].abs_()
    c.values[0][7] = 0
    blocks = -(-T // 64)
    for pool, vals in ((c.k, c.keys[0]), (c.v, c.values[0])):
        whole = torch.zeros((blocks * 64, 1, 64), dtype=c.dt)
        whole[:T] = vals
        pool[c.layer, c.table[c.rows[0], :blocks].long()] = whole.view(blocks, 64, 1, 64).transpose(1, 2)
    c.q, c.rows, c.masks = c.q.expand(n, -1, -1, -1).contiguous(), c.rows * n, [[(1 << nodes) - 1] * nodes] * n
    out, lse = c.run()
    assert c.cache.status() == 0
    ref, rl, size = D.attention(c.q[0, :1], c.keys[0], c.values[0], torch.ones((1, T), dtype=torch.bool), c.scale)
    half = D.half_step(c.dt)
    rel = (64 + 16) * 2.0 ** -24 * 17.5 + 2.0 ** -20
    small = 2.0 ** -32 * c.values[0].double().sum(0).repeat_interleave(4, 0) if dtype == "fp16" else 0.0
    assert (ref > 0.001).all()
    assert ((out.double() - ref).abs() <= half * ref * 1.02 + (half + 2 * rel) * size + small + 1e-7).all()
    assert ((lse.double() - rl).abs() <= 2 * rel + 1e-6 * rl.abs() + 1e-6).all()


@pytest.mark.parametrize("nodes,Hq,Hk,dtype", [
    (13, 16, 2, "bf16"),        # 104 rows a K head: one row tile
    (20, 16, 2, "fp16"),        # 160: two that share K and V
    (64, 8, 1, "bf16"),         # 512: four
    (5, 16, 2, "bf16"),         # 40: rows laid out twice
])
def test_trees_of_more_requests_than_the_small_table_holds(nodes, Hq, Hk, dtype):
    """100 requests at D = 128: the long table of lengths, and with more than 64 rows two V tiles in flight."""
    rng = random.Random(nodes)
    c = Case([rng.choice([0, 1, 127, 128, 129, rng.randint(2, 400)]) for _ in range(100)], nodes, Hq, Hk, 128, 16, dtype,
             seed=nodes)
    out, lse = c.run()
    c.check(out, lse)
    # an infinite value in the context of some requests
    for i in range(0, 100, 7):
        if c.lens[i] > 0:
            _place(c, i, c.lens[i] - 1, 17, float("inf"))
    out, _ = c.run()
    for i in range(100):
        hit = i % 7 == 0 and c.lens[i] > 0
        assert (out[i, ..., 17] == float("inf")).all() if hit else torch.isfinite(out[i]).all()
        assert torch.isfinite(out[i][..., :17]).all() and torch.isfinite(out[i][..., 18:]).all()


@pytest.mark.parametrize("layers", [1, 3])
def test_pools_past_two_to_the_31_elements(layers):
    """The last pages of pools of 2.3e9 elements: append, compact, copy on write, page copies and attention."""
    qb = _qb()
    pages, heads, page, dim, nodes = 70000 // layers, 4, 64, 128, 5
    gen = torch.Generator().manual_seed(layers)
    cache = qb.alloc_paged_cache(layers, pages, heads, page, dim, 3, 4)
    assert cache.k.numel() > 2 ** 31 - 10 ** 6 and layers * pages * heads * page * dim * 2 > 2 ** 32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.page_refs.fill_(1)
    cache.page_refs[pages - 8:] = 0         # the free pages are the last ones
    row, layer, total = i32([1]), layers - 1, 0
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros((512, dim), device="cuda")
    cs[:, :dim // 2] = 1.0                  # no rotation
    keys, values, q = [], [], None
    for chunk in (60, 60, 60, nodes):
        x = torch.randn((1, chunk, 3 * heads, dim), generator=gen).bfloat16().cuda()
        q = torch.empty((1, chunk, heads, dim), dtype=x.dtype, device="cuda")
        qb.qnre_cache_reserve(cache, row, i32([chunk]))
        qb.qnre_qkv_norm_rope_append(x[:, :, :heads], x[:, :, heads:2 * heads], x[:, :, 2 * heads:], w, w, cs, None, q, cache,
                                     layer, row)
        kept = list(range(0, chunk, 2)) if chunk != nodes else list(range(nodes))
        k = D.norm_rope(x[:, :, heads:2 * heads].cpu(), w.cpu(), cs.cpu(), torch.zeros((1, chunk), dtype=torch.int32), "rotate_half")
        keys.append(k[0, kept])
        values.append(x[0, kept, 2 * heads:].cpu())
        if chunk != nodes:
            qb.qnre_cache_compact(cache, row, i32([kept + [-1] * (chunk - len(kept))]), i32([len(kept)]))
            total += len(kept)
    assert cache.status() == 0 and cache.seq_lens.tolist() == [0, total, 0]
    keys, values = torch.cat(keys), torch.cat(values)
    half = D.half_step(torch.bfloat16)

    def check(r):
        at = torch.arange(total + nodes, device="cuda")
        stored = cache.k[layer, cache.block_table[r][at // page].long(), :, at % page].cpu()
        assert ((stored.double() - keys).abs() <= half * 1.01 * keys.abs() + 2.0 ** -18 * keys.abs() + 2.0 ** -25).all()
        out = torch.empty_like(q)
        qb.qnre_tree_attention(q, cache, layer, i32([r]), None, out, workspace=qb.tree_attention_workspace(q, cache))
        see = torch.ones((nodes, total + nodes), dtype=torch.bool).tril(total)
        ref, _, size = D.attention(q[0].cpu(), stored, values, see, dim ** -0.5)
        # unit norm weights: |q| = |k| = sqrt(dim) up to their rounding
        rel = (dim + 16) * 2.0 ** -24 * dim ** 0.5 * 1.01 + 2.0 ** -20
        assert ((out[0].cpu().double() - ref).abs() <= half * ref.abs() * 1.02 + (half + 2 * rel) * size + 1e-7).all()
        assert cache.status() == 0

    check(1)
    # a fork and its copy of the open page
    qb.qnre_cache_fork(cache, row, i32([2]))
    qb.qnre_cache_reserve(cache, i32([2]), i32([nodes]))
    a, b = cache.block_table[1, total // page].long(), cache.block_table[2, total // page].long()
    assert a != b and torch.equal(cache.v[layer, a, :, :total % page], cache.v[layer, b, :, :total % page])
    check(2)
    qb.qnre_cache_copy_pages(cache, b[None].int(), i32([0]))
    assert torch.equal(cache.k[layer, b], cache.k[layer, 0]) and torch.equal(cache.v[layer, b], cache.v[layer, 0])


@pytest.mark.parametrize("L", [200, 40000])
@pytest.mark.parametrize("nodes,Hq", [(1, 8), (5, 16), (16, 14), (40, 16)])
def test_infinite_values_whose_weight_is_below_any_float(L, nodes, Hq):
    """A score 200 nats above all others, at either end of rows that one CTA has or many: infinities far from it count."""
    for strong in (0, L - 1):
        c = Case([L], nodes, Hq, 2, 128, 64, "bf16", seed=4)
        T = L + nodes
        c.q[:] = 0
        c.q[..., 0] = 8.0
        c.keys[0][:] = 0
        c.keys[0][strong, :, 0] = 200.0 / (8.0 * c.scale)
        whole = torch.zeros((-(-T // 64) * 64, 2, 128), dtype=c.dt)
        whole[:T] = c.keys[0]
        c.k[1, c.table[c.rows[0], :len(whole) // 64].long()] = whole.view(-1, 64, 2, 128).transpose(1, 2)
        c.masks = [[(1 << 64) - 1 >> 64 - nodes] * nodes]
        _place(c, 0, L // 2, 5, float("inf"))
        _place(c, 0, L - 1 - strong, 100, float("-inf"))
        _place(c, 0, L, 64, float("inf"))           # the root's own draft
        out, lse = c.run()
        want = c.values[0][strong].repeat_interleave(Hq // 2, 0).expand(nodes, -1, -1).clone()
        want[..., 5], want[..., 100], want[..., 64] = float("inf"), float("-inf"), float("inf")
        assert torch.equal(out[0], want)
        assert c.cache.status() == 0
