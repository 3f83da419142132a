"""qnre_rope_table against 64-bit angles.

Tolerance: cosine and sine come out at most one unit in the last place off (2^-24 below 1), the angle, at most pi/4 after its
quarter turns, as a float (0.56 2^-24 of either), and the magnitude rounds once: 3 2^-24 of the magnitude.  A
frequency is rounded to 2^-52 relative on either side: p f 2^-50."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


def plain(n_pos, rot, first=0, theta=1e4, scaling="none", factor=1.0, original=0.0, low=1.0, high=None, magnitude=None):
    """(table, frequencies) in 64 bits, one pair at a time."""
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    freq = []
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "base":
            f = (theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == "yarn":
            pair = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        elif scaling == "wavelength":
            s = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = s * f + (1 - s) * f / factor
        freq.append(f)
    f = torch.tensor(freq, dtype=torch.float64)
    a = torch.arange(first, first + n_pos, dtype=torch.float64)[:, None] * f
    return magnitude * torch.cat([a.cos(), a.sin()], 1), f, abs(magnitude)


def check(n_pos, rot, **kw):
    qb = _qb()
    out = torch.full((n_pos + 1, rot), 7.0, device="cuda")
    qb.qnre_rope_table(out[:n_pos], **kw)
    ref, f, size = plain(n_pos, rot, **kw)
    p = torch.arange(kw.get("first", 0), kw.get("first", 0) + n_pos, dtype=torch.float64)[:, None]
    tol = size * (3 * 2.0 ** -24 + torch.cat([p * f, p * f], 1) * 2.0 ** -50)
    got = out.cpu().double()
    assert ((got[:n_pos] - ref).abs() <= tol).all(), f"worst {((got[:n_pos] - ref).abs() / tol).max():.3g} of the bound"
    assert (got[n_pos] == 7.0).all()


@pytest.mark.parametrize("n_pos", [1, 2, 31, 1000])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128])
def test_plain(n_pos, rot):
    check(n_pos, rot)


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=8.0), dict(scaling="linear", factor=0.25), dict(scaling="base", factor=4.0, theta=5e5),
    dict(scaling="yarn", factor=4.0, original=4096.0), dict(scaling="yarn", factor=16.0, original=8192.0, theta=1e6, magnitude=1.0),
    dict(scaling="yarn", factor=2.0, original=100.0, low=0.5, high=3.0), dict(scaling="wavelength", factor=8.0, original=8192.0, theta=5e5),
    dict(scaling="wavelength", factor=3.0, original=500.0, low=2.0, high=9.0), dict(magnitude=-2.5),
])
@pytest.mark.parametrize("rot", [32, 128])
def test_scaled(kw, rot):
    check(300, rot, first=100000, **kw)


@pytest.mark.parametrize("first", [0, 1 << 24, (1 << 31) - 40])
def test_far_positions(first):
    check(40, 64, first=first, theta=1e6)


def test_many_rows_and_an_empty_call():
    check(40001, 128, first=3)      # four rows a thread, a part of a block at the end
    out = torch.full((1, 16), 5.0, device="cuda")
    _qb().qnre_rope_table(out[:0])
    assert (out == 5.0).all()


def test_table_feeds_the_norm_in_a_graph():
    """Made and read in one captured graph; the norm's rotation is the table's."""
    qb = _qb()
    q, k = (torch.randn((1, 9, 2, 64), device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    table, made = torch.zeros((9, 64), device="cuda"), torch.zeros((9, 64), device="cuda")
    qo, ko, want_q, want_k = (torch.empty_like(q) for _ in range(4))
    qb.qnre_rope_table(made, scaling="linear", factor=2.0)
    qb.qnre_qk_norm_rope(q, k, w, w, made, None, want_q, want_k)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qb.qnre_rope_table(table, scaling="linear", factor=2.0)
            qb.qnre_qk_norm_rope(q, k, w, w, table, None, qo, ko)
    table.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
