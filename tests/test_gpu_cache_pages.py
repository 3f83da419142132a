"""qnre_cache_* against a list-based simulation: tables, counts, lengths and contents bit for bit."""
import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A cache on the GPU and its simulation, driven together."""

    def __init__(self, layers=2, pages=40, heads=2, page=16, dim=64, rows=8, blocks=9, dtype=torch.bfloat16, seed=0):
        from ulysses_qkv_proj_gb300 import binding as qb
        self.qb = qb
        gen = torch.Generator().manual_seed(seed)
        k, v = (torch.randn((layers, pages, heads, page, dim), generator=gen).to(dtype) for _ in range(2))
        self.cache = qb.PagedCache(k.cuda(), v.cuda(), torch.full((rows, blocks), -1, dtype=torch.int32).cuda(),
                                   torch.zeros(rows, dtype=torch.int32).cuda(),
                                   torch.zeros(pages, dtype=torch.int32).cuda())
        self.sim = D.Pages(k.clone(), v.clone(), [[-1] * blocks for _ in range(rows)], [0] * rows, [0] * pages)

    def truncate(self, rows, lens):
        self.qb.qnre_cache_truncate(self.cache, _i32(rows), _i32(lens))
        self.sim.truncate(rows, lens)

    def fork(self, src, dst):
        self.qb.qnre_cache_fork(self.cache, _i32(src), _i32(dst))
        self.sim.fork(src, dst)

    def reserve(self, rows, counts):
        self.qb.qnre_cache_reserve(self.cache, _i32(rows), _i32(counts))
        return self.sim.reserve(rows, counts)

    def compact(self, rows, paths, counts):
        width = max(len(p) for p in paths)
        full = [list(p) + [-1] * (width - len(p)) for p in paths]
        self.qb.qnre_cache_compact(self.cache, _i32(rows), _i32(full), _i32(counts))
        self.sim.compact(rows, paths, counts)

    def grow(self, rows, counts):
        """Reserve and take `counts` tokens each (their contents are whatever the pages hold)."""
        assert self.reserve(rows, counts)
        self.compact(rows, [list(range(c)) for c in counts], counts)

    def check(self, status=0):
        c = self.cache
        assert c.status() == status
        assert c.block_table.tolist() == self.sim.table
        assert c.seq_lens.tolist() == self.sim.lens
        assert c.page_refs.tolist() == self.sim.refs
        assert torch.equal(c.k.cpu(), self.sim.k) and torch.equal(c.v.cpu(), self.sim.v)


@pytest.mark.parametrize("page,dim,dtype,layers,heads", [(16, 64, torch.bfloat16, 2, 2), (8, 128, torch.float16, 1, 3),
                                                         (48, 128, torch.bfloat16, 3, 1), (64, 64, torch.float16, 1, 8)])
def test_random_walk(page, dim, dtype, layers, heads):
    import random
    rng = random.Random(page + dim)
    b = Both(layers=layers, heads=heads, page=page, dim=dim, dtype=dtype, pages=64, rows=8, blocks=9)
    for step in range(60):
        rows = rng.sample(range(8), rng.randint(1, 8))
        act = rng.choice(["step", "step", "step", "truncate", "fork", "free"])
        if act == "step":
            nodes = rng.randint(1, 20)
            rows = [r for r in rows if b.sim.lens[r] + nodes <= 9 * page]
            if not rows:
                continue
            if b.reserve(rows, [nodes] * len(rows)):
                kept = [rng.randint(0, nodes) for _ in rows]
                b.compact(rows, [sorted(rng.sample(range(nodes), c)) or [0] for c in kept], kept)
                status = 0
            else:
                status = b.qb.CACHE_NO_PAGES
        elif act == "truncate":
            b.truncate(rows, [rng.randint(0, max(1, b.sim.lens[r] + 3)) for r in rows])
            status = 0
        elif act == "free":
            b.truncate(rows[:2], [0] * len(rows[:2]))
            status = 0
        else:
            full = [r for r in range(8) if b.sim.lens[r]]
            empty = [r for r in range(8) if not b.sim.lens[r] and b.sim.table[r][0] < 0]
            if not full or not empty:
                continue
            b.fork([rng.choice(full) for _ in empty], empty)
            status = 0
        b.check(status)


def test_copy_on_write_of_the_open_page_only():
    b = Both(page=16, pages=20)
    b.grow([0], [40])
    b.fork([0, 0], [1, 2])
    b.check()
    assert b.sim.refs[b.sim.table[0][0]] == 3
    assert b.reserve([1, 2], [1, 30])
    b.check()
    assert b.sim.table[1][:2] == b.sim.table[0][:2] and b.sim.table[1][2] != b.sim.table[0][2]
    b.truncate([0, 1, 2], [0, 0, 0])
    b.check()
    assert not any(b.sim.refs)


def test_all_owners_reserve_at_once():
    """Decisions are those of the call's start: every holder copies, the old page becomes free."""
    b = Both(page=8, pages=12)
    b.grow([0], [5])
    b.fork([0], [1])
    old = b.sim.table[0][0]
    assert b.reserve([0, 1], [1, 1])
    b.check()
    assert b.sim.refs[old] == 0


def test_too_few_pages_changes_nothing():
    b = Both(page=8, pages=3)
    b.grow([0], [8])
    assert not b.reserve([0, 1], [8, 16])
    b.check(b.qb.CACHE_NO_PAGES)
    assert b.reserve([1], [16])
    b.check()
    assert not b.reserve([2], [8 * 9 + 1])                 # past max_blocks
    b.check(b.qb.CACHE_NO_PAGES)


def test_compact_overlapping_path_across_pages():
    b = Both(page=8, pages=20, blocks=6)
    b.grow([3], [6])
    assert b.reserve([3], [20])
    b.compact([3], [[1, 2, 3, 4, 8, 9, 17, 19]], [8])
    b.check()
    assert b.reserve([3, 4], [20, 20])
    b.compact([3, 4], [list(range(1, 20)), [0]], [19, 1])
    b.check()


def test_sixty_four_nodes_and_many_pages():
    b = Both(page=8, pages=20011, rows=4, blocks=30, layers=1, heads=1)
    b.cache.page_refs[:16500] = 1
    b.sim.refs[:16500] = [1] * 16500
    b.cache.page_refs[16600:20000] = 2
    b.sim.refs[16600:20000] = [2] * 3400
    b.grow([0, 1], [64, 37])
    assert b.reserve([0], [64])
    b.compact([0], [list(range(63, 64))], [1])
    b.check()
    assert b.reserve([2], [8 * 30])
    b.check()


def test_reserve_of_thousands_of_blocks():
    """Windows longer than one round of the bookkeeping, free pages far apart, a shared open block among them."""
    b = Both(page=8, pages=40003, rows=5, blocks=2600, layers=1, heads=1)
    held = torch.arange(40003) % 3 != 0
    held[30000:] = False
    b.cache.page_refs[held.nonzero()[:, 0].cuda()] = 1
    b.sim.refs = held.int().tolist()
    b.grow([1], [13])
    b.fork([1], [4])
    assert b.reserve([0, 4, 2, 3], [8 * 1024, 8 * 2500, 0, 8 * 2600])
    b.check()
    assert not b.reserve([1], [8 * 2600])                 # past max_blocks
    b.check(b.qb.CACHE_NO_PAGES)
    b.truncate([0, 1, 2, 3, 4], [0, 0, 0, 0, 0])
    b.check()


def test_misuse_is_reported():
    b = Both(page=8, pages=10)
    qb, c = b.qb, b.cache
    b.grow([0], [9])
    qb.qnre_cache_fork(c, _i32([0, 0, 7]), _i32([0, 99, -1]))
    b.check(qb.CACHE_BAD_ROW)
    qb.qnre_cache_truncate(c, _i32([8, -1]), _i32([0, 0]))
    b.check(qb.CACHE_BAD_ROW)
    qb.qnre_cache_compact(c, _i32([1]), _i32([[1, 2]]), _i32([0]))
    b.check()
    qb.qnre_cache_compact(c, _i32([5]), _i32([[2, 70]]), _i32([2]))     # no pages there
    assert c.status() == qb.CACHE_BAD_PAGE
    c.page_refs.zero_()
    c.seq_lens.zero_()
    qb.qnre_cache_truncate(c, _i32([0]), _i32([0]))
    assert c.status() == qb.CACHE_BAD_REFS and not c.page_refs.any()


def test_copy_pages_and_graph_replay():
    b = Both(page=16, pages=300, layers=3, heads=4, dim=128)
    src, dst = list(range(0, 100)), list(range(150, 250))
    b.qb.qnre_cache_copy_pages(b.cache, _i32(src), _i32(dst))
    for pool in (b.sim.k, b.sim.v):
        pool[:, dst] = pool[:, src]
    b.check()
    b.qb.qnre_cache_copy_pages(b.cache, _i32([0, 5]), _i32([300, 6]))
    for pool in (b.sim.k, b.sim.v):
        pool[:, 6] = pool[:, 5]
    b.check(b.qb.CACHE_BAD_PAGE)
    # a captured step (reserve, compact) grows the same rows on every replay
    rows, room, path, kept = _i32([0, 1]), _i32([5, 5]), _i32([[0, 2, 4], [0, 1, 3]]), _i32([3, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.qb.qnre_cache_reserve(b.cache, rows, room)
        b.qb.qnre_cache_compact(b.cache, rows, path, kept)
    for _ in range(9):
        g.replay()
        assert b.sim.reserve([0, 1], [5, 5])
        b.sim.compact([0, 1], path.tolist(), kept.tolist())
    b.check()


@pytest.mark.parametrize("length", [-1, -100, -2 ** 31])
def test_lengths_below_zero_count_as_none(length):
    """Truncate, compact, fork and reserve of a row with such a length leave the other rows' blocks alone."""
    b = Both(page=8, pages=40, rows=6, blocks=9)
    b.grow([0, 1, 2, 3, 5], [64, 60, 63, 20, 9])
    b.grow([0, 2], [6, 9])
    for call in ("truncate", "compact", "reserve"):
        b.cache.seq_lens[3] = length
        b.sim.lens[3] = 0
        if call == "truncate":
            b.truncate([3], [5])
        elif call == "compact":
            assert b.reserve([3], [4])
            b.cache.seq_lens[3] = length
            b.compact([3], [[0, 2, 3]], [3])
        else:
            assert b.reserve([3], [30])
            b.cache.seq_lens[3] = b.sim.lens[3] = 0
        b.check()
    b.truncate([3], [0])
    b.cache.seq_lens[3] = length
    b.sim.lens[3] = 0
    b.fork([3], [4])
    b.cache.seq_lens[3] = 0
    b.check()


def _append(b, rows, tokens, gen):
    """Appends `tokens` random tokens to each row in layer 0; returns what v holds."""
    heads, dim = b.sim.k.shape[2], b.sim.k.shape[4]
    n = len(rows)
    qkv = torch.randn((n, tokens, 3 * heads, dim), generator=gen).to(b.sim.k.dtype).cuda()
    q, k, v = qkv[:, :, :heads], qkv[:, :, heads:2 * heads], qkv[:, :, 2 * heads:]
    w = torch.ones(dim, dtype=qkv.dtype, device="cuda")
    out = torch.empty((n, tokens, heads, dim), dtype=qkv.dtype, device="cuda")
    b.qb.qnre_qkv_norm_rope_append(q, k, v, w, w, D.angles(256, dim).cuda(), None, out, b.cache, 0, _i32(rows))
    assert torch.isfinite(out).all()
    return v.cpu()


def test_a_refused_reserve_leaves_shared_pages_alone():
    """Two forks, no free page for their copies: their drafts go nowhere and their lengths stay."""
    b = Both(page=16, pages=2)
    b.grow([0], [20])
    b.fork([0], [1])
    b.check()
    assert not b.reserve([0, 1], [3, 3])
    b.check(b.qb.CACHE_NO_PAGES)
    gen = torch.Generator().manual_seed(1)
    _append(b, [0, 1], 3, gen)
    b.check(b.qb.CACHE_BAD_PAGE)
    for path in ([0, 1, 2], [0, 2, -1], [1, 2, -1]):
        b.qb.qnre_cache_compact(b.cache, _i32([0, 1]), _i32([path, path]), _i32([2, 2]))
        b.check(b.qb.CACHE_BAD_PAGE)
    # with the other row gone the page is this row's own again
    b.truncate([1], [0])
    v = _append(b, [0], 3, gen)
    assert b.cache.status() == 0
    page = b.sim.table[0][1]
    for s in range(3):
        assert torch.equal(b.cache.v[0, page, :, 4 + s].cpu(), v[0, s])
    b.qb.qnre_cache_compact(b.cache, _i32([0]), _i32([[0, 2, -1]]), _i32([2]))
    assert b.cache.status() == 0 and b.cache.seq_lens.tolist()[:2] == [22, 0]
    assert torch.equal(b.cache.v[0, page, :, 5].cpu(), v[0, 2])


def test_append_skips_the_shared_page_and_fills_the_next():
    """A shared open page and an own one behind it: only the own one takes its tokens."""
    b = Both(page=8, pages=4, layers=1)
    b.grow([0], [13])
    b.fork([0], [1])
    own = 3
    b.cache.block_table[1, 2] = own
    b.cache.page_refs[own] = 1
    before = b.cache.v.cpu().clone()
    v = _append(b, [1], 6, torch.Generator().manual_seed(2))
    assert b.cache.status() == b.qb.CACHE_BAD_PAGE
    after = b.cache.v.cpu()
    for s in range(3):
        assert torch.equal(after[0, own, :, s], v[0, 3 + s])
    after[0, own, :, :3] = before[0, own, :, :3]
    assert torch.equal(after, before)


@pytest.mark.parametrize("path,kept", [([0, 1, 2, 3, 4], 2), ([0, 1, 3, 4, 5], 2), ([0, 2, 3, 4, 5], 1), ([2, 3, 4, 5, 6], 0),
                                       ([1, 2, 3, 4, 5], 1), ([0, 1], 2)])
@pytest.mark.parametrize("layers", [1, 8])
def test_lengths_stay_within_the_pages_a_row_holds(path, kept, layers):
    """Two more slots in the last page and none behind it: tokens that would lie, or come from, past it are not kept."""
    b = Both(page=8, pages=8, blocks=3, layers=layers, heads=4)
    b.grow([0, 2], [14, 9])
    assert b.reserve([0], [2])
    listed = len(path)
    b.qb.qnre_cache_compact(b.cache, _i32([0, 2]), _i32([path, [0] * listed]), _i32([listed, 0]))
    b.sim.compact([0, 2], [path[:kept], []], [kept, 0])
    b.check(b.qb.CACHE_BAD_PAGE if kept < listed else 0)


def test_lengths_stay_within_the_table():
    b = Both(page=8, pages=20, blocks=3)
    b.grow([1], [22])
    assert b.reserve([1], [2])
    b.qb.qnre_cache_compact(b.cache, _i32([1]), _i32([list(range(40))]), _i32([40]))
    b.sim.compact([1], [[0, 1]], [2])
    b.check(b.qb.CACHE_BAD_PAGE)
