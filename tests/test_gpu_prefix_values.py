"""What one request's values do to the others in qnre_prefix_attention: nothing, bit for bit.

Rows of many requests share a tile's products, so infinite and NaN values, scores beyond the cap and what lies in unused slots must
stay with the rows that see them.  Tolerance against the 64-bit form: as in test_gpu_prefix_attention, but a capped score that lies
below the cap is off by the roundings of its polynomial alone, four of 2^-24 of the score."""
import pytest
import torch

import _decode as D
from test_gpu_prefix_attention import Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def check_closely(c, out, lse, only, columns=None):
    """Rows of requests `only` against the plain form, scores below the cap; columns: [Hq, dim] of those to compare."""
    half, dim = D.half_step(c.dt), c.q.shape[-1]
    for i in only:
        ref, rl, size, bias = c.plain(i)
        s = float(c.q[i].double().norm(dim=-1).max() * c.keys[i].double().norm(dim=-1).max() * c.scale)
        assert not c.cap or s < c.cap
        rel = (dim + 16) * 2.0 ** -24 * s + 2.0 ** -20 + 4 * 2.0 ** -24 * s + 4 * 2.0 ** -24 * bias
        tol = half * ref.abs() * 1.02 + (half + 2 * rel) * size + 1e-7
        err = (out[i].double() - ref).abs()
        if columns is not None:
            err, tol = err[:, columns], tol[:, columns]
        assert (err <= tol).all(), f"request {i}: worst excess {(err - tol).max():.3g}"
        assert ((lse[i].double() - rl).abs() <= 2 * rel + 1e-6 * rl.abs() + 1e-6).all()


# requests of a unit: 32, 128 (marks by pairs), 16, 2 (63 rows each), 1 (units of nodes), 9 heads over three quarters
UNITS = [dict(Hq=4, Hk=1), dict(Hq=2, Hk=2), dict(Hq=8, Hk=1), dict(Hq=7, Hk=1, nodes=9), dict(Hq=8, Hk=1, nodes=20), dict(Hq=9, Hk=1, nodes=3)]


@pytest.mark.parametrize("kw", UNITS)
@pytest.mark.parametrize("dim,dtype,grouped", [(128, "bf16", True), (64, "fp16", False), (64, "bf16", True), (128, "fp16", False)])
def test_infinite_values_leave_other_columns_and_requests(kw, dim, dtype, grouped):
    """An infinite V in a request's own context, and one in a draft: everything that does not see it keeps its bits, what sees it
    is infinite in that column alone."""
    c = Case([(3, 160), (2, 64)], [150, 40, 3, 200], dim=dim, dtype=dtype, seed=30, alone=2, **kw)
    N, G = c.nodes, c.q.shape[2] // c.Hk
    want, want_lse = c.run(groups=grouped)
    i, last = 4, c.Hk - 1
    x, y = c.lens[i] - 2, c.lens[6] + N - 1           # request 4's context, request 6's last draft
    c.values[i][x, last, 7], c.values[i][x, last, 9], c.values[i][x - 1, last, 9] = INF, INF, -INF
    c.values[i][c.lens[i] - 1, last, dim - 1] = -INF
    c.values[6][y, last, 3] = NAN
    c.fill()
    out, lse = c.run(groups=grouped)
    assert c.cache.status() == 0 and torch.equal(lse, want_lse)
    heads = slice(last * G, (last + 1) * G)
    assert (out[i, :, heads, 7] == INF).all() and out[i, :, heads, 9].isnan().all() and (out[i, :, heads, dim - 1] == -INF).all()
    for column in (7, 9, dim - 1):
        want[i, :, heads, column] = out[i, :, heads, column] = 0
    for t in range(N):
        if c.masks[6][t] >> (N - 1) & 1:
            assert out[6, t, heads, 3].isnan().all()
            want[6, t, heads, 3] = out[6, t, heads, 3] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("kw", UNITS)
@pytest.mark.parametrize("bad", [NAN, INF])
def test_strange_keys_leave_other_requests(kw, bad):
    c = Case([(3, 160), (2, 64)], [150, 40, 3, 200], seed=31, alone=2, **kw)
    want, want_lse = c.run()
    c.keys[4][c.lens[4] - 2, c.Hk - 1] = bad
    c.fill()
    out, lse = c.run()
    others = [j for j in range(c.n) if j != 4]
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])


@pytest.mark.parametrize("cap,slopes", [(30.0, False), (1e6, False), (1e30, False), (1e4, True), (0.0, True)])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_infinite_values_under_caps_and_biases(cap, slopes, dim, dtype):
    """The rows that see an infinite V, and their neighbours, against 64 bits."""
    c = Case([(4, 160), (2, 48)], [90, 3, 30], nodes=3, Hq=4, Hk=2, dim=dim, dtype=dtype, cap=cap, slopes=slopes, seed=32, alone=1)
    c.values[2][c.common[2] + 1, 0, 5] = INF
    c.values[3][c.lens[3], 1, 6] = INF                # the root of request 3's drafts, which all its nodes see
    c.values[1][20, 1, 8] = -INF                      # in the first group's common tokens
    for j in range(1, 5):
        c.values[j][20] = c.values[1][20]
    c.fill()
    out, lse = c.run()
    assert (out[2, :, :2, 5] == INF).all() and (out[3, :, 2:, 6] == INF).all() and (out[1:5, :, 2:, 8] == -INF).all()
    for v in c.values:
        v[~torch.isfinite(v)] = 0
    columns = torch.ones(c.q.shape[2:], dtype=torch.bool)
    columns[:2, 5] = columns[2:, 6] = columns[2:, 8] = False
    check_closely(c, out, lse, range(c.n), columns)


@pytest.mark.parametrize("cap", [1e4, 30.0])
@pytest.mark.parametrize("kw", [dict(Hq=7, Hk=1, nodes=5), dict(Hq=4, Hk=2, nodes=2, dim=64, dtype="fp16"), dict(Hq=14, Hk=2, nodes=1)])
def test_unused_slots_do_not_choose_the_arithmetic(cap, kw):
    """K in slots behind a row's tokens: zeros, or values far beyond the cap; the same bits, and as near as scores that small come."""
    c = Case([(5, 96), (3, 32)], [21, 3, 130], cap=cap, seed=33, alone=1, **kw)
    unused = torch.isnan(c.k)
    got = []
    for filling in (0.0, 3000.0):
        c.k[unused] = filling
        got.append(c.run())
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    if cap > 100:
        check_closely(c, *got[1], range(c.n))


@pytest.mark.parametrize("cap", [1e4, 50.0])
@pytest.mark.parametrize("grouped", [True, False])
def test_scores_beyond_the_cap_stay_with_their_row(cap, grouped):
    """One request's queries grow until its scores pass the cap; the others keep their bits."""
    c = Case([(6, 160), (3, 64)], [21, 3, 130], nodes=2, Hq=4, Hk=2, cap=cap, seed=34)
    want, want_lse = c.run(groups=grouped)
    c.q[2] *= 4 * cap
    out, lse = c.run(groups=grouped)
    others = [j for j in range(c.n) if j != 2]
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])
    c.check(out, lse, only=[2])


@pytest.mark.parametrize("cap", [1e4, 30.0])
def test_hidden_drafts_do_not_choose_the_arithmetic(cap):
    """One draft's K grows far beyond the cap; the nodes whose masks do not name it keep their bits."""
    c = Case([(4, 96)], [21, 3], nodes=9, Hq=4, Hk=2, cap=cap, slopes=True, seed=35)
    want, want_lse = c.run()
    c.keys[1][c.lens[1] + 2] *= 1e4
    c.fill()
    out, lse = c.run()
    sees = [m >> 2 & 1 for m in c.masks[1]]
    assert 0 < sum(sees) < 9
    for i in range(c.n):
        rows = [t for t in range(9) if i != 1 or not sees[t]]
        assert torch.equal(out[i, rows], want[i, rows]) and torch.equal(lse[i, rows], want_lse[i, rows])
    c.check(out, lse, only=[1])
