"""qnre_sample and qnre_filter_probs against a sorted 64-bit evaluation.

Tokens and the set of tokens kept have to be equal.  A probability is formed from 31 bits of its weight (2^-30), as a float
(2^-24), times the total's reciprocal as a float (2^-24), rounded (2^-24): within 4 2^-24, and 2^-148 where it is denormal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BIG = float(np.finfo(np.float32).max)


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


def weights(x, T, k, p, m):
    """Kept weights of one row (float64 numpy), zero for the rest; None where there is no token."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, BIG)).astype(np.float64)
    V = len(x)
    if x.max() == -np.inf:
        return None
    if not T > 0:
        w = np.zeros(V)
        w[x.argmax()] = 1
        return w
    order = np.argsort(-x, kind="stable")
    w = np.exp((x[order] - x.max()) / T)
    keep = x[order] > -np.inf
    if m > 0:
        keep &= x[order] >= x.max() + T * np.log(min(m, 1.0))
    if 0 < k < V:
        keep[k:] = False
    w = np.where(keep, w, 0)
    if p < 1:
        w = np.where((np.cumsum(w) - w < max(p, 0.0) * w.sum()) | (np.arange(V) == 0), w, 0)
        keep &= w > 0
    out = np.zeros(V)
    out[order] = np.where(keep, w, 0)
    return out


def token(w, u):
    if w is None:
        return -1
    c = np.cumsum(w)
    u = 0.0 if not u > 0 else u
    over = np.nonzero((c > u * c[-1]) & (w > 0))[0]
    return int(over[0]) if len(over) and u < 1 else int(np.nonzero(w)[0].max())


def settings(n, T=1.0, k=0, p=1.0, m=0.0):
    row = lambda x, t: torch.tensor(x if isinstance(x, list) else [x] * n, dtype=t, device="cuda")
    return dict(temperature=row(T, torch.float32), top_k=row(k, torch.int32), top_p=row(p, torch.float32), min_p=row(m, torch.float32))


def check(logits, u=None, **kw):
    """Both calls on logits [n, V]; rows' settings by keyword (one value or a list)."""
    qb = _qb()
    n, V = logits.shape
    s = settings(n, **kw)
    if u is None:
        u = torch.rand(n, generator=torch.Generator().manual_seed(V + n)).cuda()
    tokens = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((n, 1, V), 3.0, device="cuda")
    qb.qnre_sample(logits, u, tokens, **s)
    qb.qnre_filter_probs(logits[:, None], probs, **s)
    got, x, us = probs.cpu().numpy()[:, 0], logits.float().cpu().numpy(), u.double().cpu().numpy()
    host = [t.double().cpu().numpy() for t in s.values()]
    for i in range(n):
        w = weights(x[i], host[0][i], int(host[1][i]), host[2][i], host[3][i])
        assert int(tokens[i]) == token(w, us[i]), f"row {i}"
        if w is None:
            assert not got[i].any()
            continue
        e = w / w.sum()
        assert (np.abs(got[i] - e) <= 4 * 2.0 ** -24 * e + 2.0 ** -148).all(), f"row {i}"
        assert ((got[i] > 0) == (e > 2.0 ** -140))[(e == 0) | (e > 2.0 ** -140)].all(), f"row {i}: kept"
    return tokens, probs


def bell(n, V, dtype="fp32", seed=0, spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((n, V), generator=gen) * spread
    return x.to(DT[dtype]).cuda()


@pytest.mark.parametrize("V", [1, 2, 7, 33, 1023, 1024, 1025, 4096, 9000, 40003])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_every_setting(V, dtype):
    T = [0.0, 1.0, 0.7, 1.0, 0.9, 1.4, 0.5, 1.0, -1.0, 0.05, 30.0]
    k = [5, 0, 50, 0, 0, 40, 1, 3000, 2, 0, 0]
    p = [0.5, 1.0, 1.0, 0.9, 1.0, 0.95, 0.3, 0.99, 0.9, 0.999, 0.6]
    m = [0.5, 0.0, 0.0, 0.0, 0.05, 0.02, 0.0, 0.0, 0.0, 0.0, 0.0]
    check(bell(len(T), V, dtype, seed=V), T=T, k=k, p=p, m=m)


@pytest.mark.parametrize("n,V,dtype", [(1, 131075, "fp32"), (40, 131075, "bf16"), (3, 262147, "fp32"), (2, 1 << 20, "fp16"), (1, 1 << 20, "fp32"),
                                       (700, 3001, "fp32"), (1300, 1100, "bf16")])
def test_cluster_sizes(n, V, dtype):
    """From sixteen CTAs a row down to one, rows held in shared memory and rows read again."""
    cycle = lambda x: [x[i % len(x)] for i in range(n)]
    check(bell(n, V, dtype, seed=n), T=cycle([0.8, 1.0, 1.3]), k=cycle([0, 50, 0, 2000, 0]), p=cycle([0.9, 1.0, 0.99, 0.95]),
          m=cycle([0.0, 0.0, 0.01]))


@pytest.mark.parametrize("n,V,dtype", [(306, 26000, "bf16"), (306, 26000, "fp32"), (9, 26001, "fp16"), (18, 900, "fp32")])
def test_a_top_p_cut_lies_anywhere(n, V, dtype):
    """Also where the counts leave more bins than the window has (a cut in a gap of logits far apart, few levels)."""
    p = [0.0, 1e-6, 0.01, 0.3, 0.5, 0.8, 0.9, 0.99, 0.9999]
    T = [1.0, 0.3, 2.5, 0.7]
    x = bell(n, V, dtype, seed=V + n)
    x[1::3] = x[1::3] * 4
    x[2::6] = torch.round(x[2::6])
    check(x, p=[p[i % 9] for i in range(n)], T=[T[i // 9 % 4] for i in range(n)])


@pytest.mark.parametrize("levels", [1, 2, 5, 60])
@pytest.mark.parametrize("V", [500, 5000, 70000])
def test_ties_go_by_index(levels, V):
    """Few values: cuts fall among thousands of equal logits, beyond what a list holds."""
    gen = torch.Generator().manual_seed(levels + V)
    x = (torch.randint(0, levels, (6, V), generator=gen).float() * 0.37 - 3).cuda()
    check(x, T=[1.0, 0.8, 1.0, 2.0, 1.0, 0.0], k=[0, V // 3, V // 7, 0, 3, 0], p=[0.5, 1.0, 0.77, 0.9, 1.0, 1.0])


def test_logits_far_apart():
    """Values beyond the bins' range on both sides of a cut, and steps of every size."""
    gen = torch.Generator().manual_seed(4)
    base = torch.cat([torch.randn(3000, generator=gen) * 1e-4, torch.randn(3000, generator=gen) * 50, -torch.rand(3000, generator=gen) * 1e6,
                      torch.randn(3000, generator=gen) * 1e-30])
    x = torch.stack([base[torch.randperm(12000, generator=gen)] for _ in range(6)]).cuda()
    check(x, T=[1.0, 100.0, 1e4, 1e6, 3.0, 1e-3], k=[5000, 0, 7001, 0, 11000, 0], p=[1.0, 0.9, 0.5, 0.999, 0.99, 0.9])


def test_masked_and_strange_values():
    V = 3000
    x = bell(9, V, seed=8)
    lowest = torch.finfo(torch.float32).min
    x[0, 10:] = lowest                  # a mask of the type's lowest value
    x[1, :] = lowest                    # all of it
    x[2, :] = -float("inf")             # no token
    x[3, 1::2] = -float("inf")
    x[4, ::3] = float("nan")
    x[5, 7] = x[5, 11] = float("inf")
    x[6, :] = float("nan")
    x[7, :-1] = -float("inf")
    x[8, :] = 0.0
    x[8, ::2] = -0.0                    # one value
    for kw in (dict(), dict(k=4), dict(p=0.8), dict(k=100, p=0.5, m=0.1), dict(T=0.0), dict(m=1.0)):
        check(x, **kw)
    for dtype in ("bf16", "fp16"):
        y = bell(3, V, dtype, seed=9)
        y[0, 5:] = torch.finfo(DT[dtype]).min
        y[1, ::2] = -float("inf")
        y[2, 3] = float("inf")
        check(y, p=0.9)


@pytest.mark.parametrize("kw", [dict(p=0.0), dict(p=-1.0), dict(p=1e-7), dict(p=float("nan")), dict(k=-3), dict(k=2 ** 31 - 1), dict(m=5.0),
                                dict(m=-1.0), dict(m=float("nan")), dict(T=float("nan")), dict(T=1e-30), dict(T=1e30), dict(T=1e-45),
                                dict(T=float("inf")), dict(k=1, p=0.0, m=1.0)])
def test_ends_of_the_settings(kw):
    check(bell(4, 2500, seed=3), **kw)


def test_random_numbers_at_the_ends():
    n = 9
    u = torch.tensor([0.0, 1e-45, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), 1e-8]).cuda()
    for kw in (dict(), dict(k=3), dict(p=0.9)):
        check(bell(1, 2000, seed=5).expand(n, -1), u=u, **kw)


def test_every_share_of_a_row_is_drawn_as_often_as_its_weight():
    """A grid of numbers over one row: each token as often as its weight says, to one step of the grid."""
    qb = _qb()
    n, V = 4000, 50
    x = bell(1, V, seed=6).expand(n, -1)
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().cuda()
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    qb.qnre_sample(x, u, tokens, **settings(n, p=0.9))
    w = weights(x[0].cpu().numpy(), 1.0, 0, float(np.float32(0.9)), 0.0)
    seen = np.bincount(tokens.cpu().numpy(), minlength=V)
    assert (np.abs(seen - n * w / w.sum()) <= 1.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_of_a_wider_tensor(dtype):
    """Rows that begin anywhere: the columns of a padded projection, the last node of each tree, rows read twice."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.randn((5, 3, 4100), generator=gen, device="cuda").to(DT[dtype])
    for at in range(1, 9):
        check(wide[:, 1, at:at + 4001], k=[0, 5, 0, 600, 0], p=[1.0, 0.9, 0.95, 1.0, 0.5])
    check(wide[0, 0, 3:1003].expand(4, -1), p=0.7)
    check(wide[:, 0, 17:18], p=0.7)


def test_filter_serves_trees():
    """Rows of a request share its settings; views of trees; the rest of the output stays as it was."""
    qb = _qb()
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, N, V = 3, 5, 777
    big = torch.randn((n, N + 2, V + 9), generator=gen, device="cuda").bfloat16() * 3
    x = big[:, 1:1 + N, 4:4 + V]
    s = settings(n, T=[0.7, 0.0, 1.2], k=[20, 0, 0], p=[1.0, 1.0, 0.9], m=[0.0, 0.0, 0.05])
    room = torch.full((n * N * V + 8,), 9.0, device="cuda")
    out = room[4:-4].view(n, N, V)
    qb.qnre_filter_probs(x, out, **s)
    assert (room[:4] == 9).all() and (room[-4:] == 9).all()
    for i in range(n):
        for j in range(N):
            w = weights(x[i, j].float().cpu().numpy(), *(float(s[k][i]) for k in ("temperature",)), int(s["top_k"][i]),
                        float(s["top_p"][i]), float(s["min_p"][i]))
            e = w / w.sum()
            g = out[i, j].cpu().numpy()
            assert ((g > 0) == (e > 0)).all() and (np.abs(g - e) <= 4 * 2.0 ** -24 * e).all()


def test_no_settings_and_no_rows():
    qb = _qb()
    x, u = bell(3, 100), torch.rand(3, device="cuda")
    a, b = (torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2))
    qb.qnre_sample(x, u, a)
    qb.qnre_sample(x, u, b, **settings(3))
    assert torch.equal(a, b)
    qb.qnre_sample(x[:0], u[:0], a[:0])
    assert torch.equal(a, b)


def test_replayed_and_on_two_streams():
    """Captured once and replayed on new logits, while another stream works: the same tokens as call by call."""
    qb = _qb()
    n, V = 20, 30001
    s = settings(n, T=0.8, k=[0, 40] * 10, p=0.9)
    x, y = bell(n, V, seed=1), bell(n, V, "bf16", seed=2)
    u = torch.rand(n, device="cuda")
    tokens, other = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    probs = torch.empty((n, 1, V), device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=one):
            qb.qnre_sample(x, u, tokens, **s)
            qb.qnre_filter_probs(x[:, None], probs, **s)
    for seed in (11, 12):
        x.copy_(bell(n, V, seed=seed))
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            g.replay()
        for _ in range(3):
            qb.qnre_sample(y, u, other, stream=two, **s)
        torch.cuda.synchronize()
        want_t, want_p = check(x, u=u, T=0.8, k=[0, 40] * 10, p=0.9)
        assert torch.equal(tokens, want_t) and torch.equal(probs, want_p)
        want, _ = check(y, u=u, T=0.8, k=[0, 40] * 10, p=0.9)
        assert torch.equal(other, want)


def test_filtered_probabilities_verify_a_tree():
    """qnre_verify_tree on filtered probabilities: drafts outside the kept set are refused, and the emitted token is the one that
    qnre_sample draws from the same logits with the same number."""
    qb = _qb()
    n, V = 64, 999
    x = bell(n, V, seed=21)
    s = settings(n, T=0.9, k=20, p=0.9)
    probs = torch.empty((n, 2, V), device="cuda")
    both = torch.stack([x, bell(n, V, seed=22)], 1)
    qb.qnre_filter_probs(both, probs, **s)
    outside = (probs[:, 0] == 0).int().argmax(-1).int()
    toks = torch.stack([torch.zeros_like(outside), outside], 1).contiguous()
    parents = torch.tensor([[-1, 0]] * n, dtype=torch.int32, device="cuda")
    u = torch.rand(n, device="cuda")
    path, counts, following, tokens = (torch.empty(shape, dtype=torch.int32, device="cuda") for shape in ((n, 2), (n,), (n,), (n,)))
    qb.qnre_verify_tree(probs, None, toks, parents, torch.zeros((n, 2), device="cuda"), u, path, counts, following)
    qb.qnre_sample(x, u, tokens, **s)
    assert (counts == 1).all()
    # (the probabilities are rounded to floats: a draw within 20 roundings of a border may differ)
    e = probs[:, 0].double().cpu().numpy()
    differ = (following != tokens).nonzero()[:, 0].tolist()
    for i in differ:
        c = np.cumsum(e[i])
        assert np.abs(c - float(u[i]) * c[-1]).min() < 40 * 2.0 ** -24
    assert len(differ) <= 1
