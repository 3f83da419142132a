"""qnre_verify_tree and qnre_tree_masks: integers equal to a one-number-at-a-time 64-bit walk."""
import random

import numpy as np
import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu


def _run(p, q, tokens, parents, accept, sample, node_counts=None):
    from ulysses_qkv_proj_gb300 import binding as qb
    n, N, V = p.shape
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()
    f32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().cuda()
    path = torch.full((n, N), 77, dtype=torch.int32, device="cuda")
    kept, nxt = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    qb.qnre_verify_tree(f32(p), None if q is None else f32(q), i32(tokens), i32(parents), f32(accept), f32(sample), path,
                        kept, nxt, node_counts=None if node_counts is None else i32(node_counts))
    return path.tolist(), kept.tolist(), nxt.tolist()


def _check(p, q, tokens, parents, accept, sample, node_counts=None):
    got = _run(p, q, tokens, parents, accept, sample, node_counts)
    for b in range(len(p)):
        up = list(parents[b])
        if node_counts is not None:
            up = up[:node_counts[b]] + [-1] * (len(up) - node_counts[b])
        path, nxt = D.verify(p[b], None if q is None else q[b], tokens[b], up, accept[b], sample[b])
        assert got[0][b] == path + [-1] * (len(up) - len(path)), f"request {b}"
        assert got[1][b] == len(path) and got[2][b] == nxt, f"request {b}: {got[2][b]} for {nxt}"
    return got


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _inputs(n, N, V, branch, seed, near=1.0):
    rng = np.random.default_rng(seed)
    pr = random.Random(seed)
    base = rng.standard_normal((n, N, V)) * 2
    p, q = _softmax(base), _softmax(base + near * rng.standard_normal((n, N, V)))
    parents = [D.random_tree(pr, N, branch) for _ in range(n)]
    tokens = [[int(rng.choice(V, p=q[b, max(u, 0)].astype(np.float64) / q[b, max(u, 0)].sum(dtype=np.float64)))
               for u in parents[b]] for b in range(n)]
    return p, q, tokens, parents, rng.random((n, N)).astype(np.float32), rng.random(n).astype(np.float32)


@pytest.mark.parametrize("n,N,V,branch", [(1, 1, 1, 1), (3, 2, 7, 1), (5, 9, 33, 2), (17, 64, 1000, 3), (4, 5, 4099, 1),
                                          (2, 33, 50021, 4), (80, 6, 40000, 2), (200, 4, 9001, 2)])
def test_walks(n, N, V, branch):
    p, q, *rest = _inputs(n, N, V, branch, n + N + V)
    got = _check(p, q, *rest)
    _check(p, None, *rest)
    if n * N > 100:
        assert len(set(got[1])) > 2     # short and long paths both occur


def test_identical_distributions_accept_everything():
    p, _, tokens, parents, u, s = _inputs(6, 8, 500, 1, 1)
    parents = [[-1] + list(range(7))] * 6
    tokens = [[0] + [int(np.argmax(p[b, i - 1])) for i in range(1, 8)] for b in range(6)]
    path, kept, _ = _check(p, p.copy(), tokens, parents, u, s)
    assert kept == [8] * 6


def test_borders():
    """Greedy rows, drafts with no target mass, everything rejected, nothing left, equal siblings, empty rows."""
    V = 100
    one = lambda x: np.eye(V, dtype=np.float32)[x]
    half = 0.5 * (one(3) + one(90))
    p = np.stack([np.stack(r) for r in [
        [one(5), one(6), one(7), one(8)],          # greedy: 5 accepted, then 6 against a draft of 9
        [half, one(1), one(2), one(3)],            # two children of one token: the second must see what is left
        [np.zeros(V, np.float32)] * 4,             # no mass anywhere
        [one(5), one(6), one(7), one(8)],          # draft equals target but its token has no mass in either
    ]])
    q = np.stack([np.stack(r) for r in [
        [one(5), one(9), one(7), one(8)],
        [half, half, half, half],
        [one(1)] * 4,
        [one(5), one(6), one(7), one(8)],
    ]])
    tokens = [[0, 5, 9, 7], [0, 3, 3, 90], [0, 1, 1, 1], [0, 50, 50, 5]]
    parents = [[-1, 0, 1, 2], [-1, 0, 0, 0], [-1, 0, 0, 0], [-1, 0, 0, 0]]
    for u in (0.0, 0.5, np.float32(1 - 2.0 ** -24)):
        for s in (0.0, 0.25, 0.5, np.float32(1 - 2.0 ** -24)):
            acc, smp = np.full((4, 4), u, np.float32), np.full(4, s, np.float32)
            got = _check(p, q, tokens, parents, acc, smp)
            assert got[2][2] == -1
            _check(p, None, tokens, parents, acc, smp)


def test_bad_nodes_are_left_out_and_counts_cut():
    p, q, tokens, parents, u, s = _inputs(4, 8, 300, 2, 3)
    tokens[0][1], tokens[0][2] = -1, 300
    parents[1][3], parents[1][4], parents[2][1] = 5, 4, -7
    _check(p, q, tokens, parents, u, s)
    _check(p, None, tokens, parents, u, s, node_counts=[1, 3, 8, 0])


def test_strided_rows_and_unaligned_vocabulary():
    from ulysses_qkv_proj_gb300 import binding as qb
    n, N, V = 3, 4, 5003
    p, q, tokens, parents, u, s = _inputs(n, N, V, 2, 5)
    buf = torch.zeros((N, n, V + 6), device="cuda")
    pv = buf.transpose(0, 1)[:, :, 3:3 + V]
    pv.copy_(torch.from_numpy(p))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()
    out = [torch.empty((n, N), dtype=torch.int32).cuda(), torch.empty(n, dtype=torch.int32).cuda(),
           torch.empty(n, dtype=torch.int32).cuda()]
    qb.qnre_verify_tree(pv, torch.from_numpy(q).cuda(), i32(tokens), i32(parents), torch.from_numpy(u).cuda(),
                        torch.from_numpy(s).cuda(), *out)
    want = _run(p, q, tokens, parents, u, s)
    assert [t.tolist() for t in out] == [*want]


def test_emitted_tokens_follow_the_target():
    """One drafted token, many random numbers: the first emitted token is distributed as the target's row."""
    V, n = 8, 40000
    rng = np.random.default_rng(0)
    p0, q0, p1 = (_softmax(rng.standard_normal(V)) for _ in range(3))
    p = np.broadcast_to(np.stack([p0, p1, p1]), (n, 3, V))
    q = np.broadcast_to(np.stack([q0, q0, q0]), (n, 3, V))
    x = rng.choice(V, size=(n, 2), p=q0.astype(np.float64) / q0.sum(dtype=np.float64))
    tokens = np.concatenate([np.zeros((n, 1), np.int64), x], 1)
    parents = np.broadcast_to(np.array([-1, 0, 0]), (n, 3))
    path, kept, nxt = _run(p, q, tokens, parents, rng.random((n, 3)), rng.random(n))
    first = [tokens[b][path[b][1]] if kept[b] > 1 else nxt[b] for b in range(n)]
    freq = np.bincount(first, minlength=V) / n
    # six standard deviations of a frequency over n draws
    assert (np.abs(freq - p0) <= 6 * np.sqrt(p0 * (1 - p0) / n)).all()


@pytest.mark.parametrize("n,N", [(1, 1), (7, 33), (50, 64)])
def test_masks(n, N):
    from ulysses_qkv_proj_gb300 import binding as qb
    rng = random.Random(n)
    parents = [D.random_tree(rng, N, rng.randint(1, 4)) for _ in range(n)]
    if N > 5:
        parents[0][3], parents[0][4] = 3, 9        # not earlier nodes: roots
    masks = torch.zeros((n, N), dtype=torch.int64, device="cuda")
    depths = torch.zeros((n, N), dtype=torch.int32, device="cuda")
    par = torch.tensor(parents, dtype=torch.int32).cuda()
    qb.qnre_tree_masks(par, masks, depths)
    want = [D.ancestors(p) for p in parents]
    assert torch.equal(masks.cpu(), D.signed([w[0] for w in want]))
    assert depths.tolist() == [w[1] for w in want]
    qb.qnre_tree_masks(par, depths=depths)
    qb.qnre_tree_masks(par, masks)


def test_replay_from_a_graph():
    from ulysses_qkv_proj_gb300 import binding as qb
    n, N, V = 6, 9, 20011
    args = [_inputs(n, N, V, 2, seed) for seed in (11, 12)]
    dev = lambda a: [torch.from_numpy(np.ascontiguousarray(a[0])).cuda(), torch.from_numpy(np.ascontiguousarray(a[1])).cuda(),
                     torch.tensor(a[2], dtype=torch.int32).cuda(), torch.tensor(a[3], dtype=torch.int32).cuda(),
                     torch.from_numpy(a[4]).cuda(), torch.from_numpy(a[5]).cuda()]
    first, second = dev(args[0]), dev(args[1])
    out = [torch.empty((n, N), dtype=torch.int32).cuda(), torch.empty(n, dtype=torch.int32).cuda(),
           torch.empty(n, dtype=torch.int32).cuda()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qb.qnre_verify_tree(*first, *out)
    for a, b in zip(first, second):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert [t.tolist() for t in out] == [*_run(*args[1])]
