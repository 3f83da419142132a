"""Refusals of the rotary table, shared-prefix and sampling calls: status codes before anything reaches a GPU."""
import ctypes
import math

import pytest

from test_decode_host import A, MB, CACHE_BAD, _Stream, cache, lib, view  # noqa: F401
from ulysses_qkv_proj_gb300 import binding as qb

NAN, INF = math.nan, math.inf


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), 1), (dict(out=A + 4), 3), (dict(n=-1), 1), (dict(n=0, out=None), 0), (dict(rot=0), 1), (dict(rot=24), 1),
    (dict(rot=-16), 1), (dict(rot=144), 2), (dict(first=-1), 1), (dict(first=(1 << 31) - 4), 5), (dict(n=1 << 32), 5),
    (dict(theta=1.0), 1), (dict(theta=NAN), 1), (dict(theta=INF), 1), (dict(kind=-1), 1), (dict(kind=5), 1),
    (dict(kind=1, factor=0.0), 1), (dict(kind=2, factor=-2.0), 1), (dict(kind=3, factor=NAN), 1), (dict(kind=3, original=0.0), 1),
    (dict(kind=3, low=4.0, high=4.0), 1), (dict(kind=4, low=0.0), 1), (dict(kind=4, original=INF), 1), (dict(magnitude=NAN), 1),
    (dict(kind=2, factor=1e300, theta=1e300), 1),
])
def test_table_arguments(lib, kw, want):
    f = dict(out=A, n=8, rot=64, first=0, theta=1e4, kind=0, factor=2.0, original=4096.0, low=1.0, high=32.0, magnitude=1.0)
    f.update(kw)
    s = qb._RopeScaling(*[f[k] for k in ("kind", "factor", "original", "low", "high", "magnitude")])
    assert lib.qnre_rope_table(f["out"], f["n"], f["rot"], f["first"], f["theta"], ctypes.byref(s), None) == want


SAMPLE_BAD = [
    (dict(n=-1), 1), (dict(vocab=0), 1), (dict(vocab=-5), 1), (dict(s0=-1), 1), (dict(dtype=3), 2), (dict(dtype=-1), 2),
    (dict(vocab=qb.MAX_VOCAB + 1), 5), (dict(n=(1 << 20) + 1), 5), (dict(s0=1 << 41), 5), (dict(logits=None), 1),
    (dict(out=None), 1), (dict(logits=A + 1), 3), (dict(logits=A + 2, dtype=2), 3), (dict(out=A + 10 * MB + 2), 3),
    (dict(t=A + 2), 3), (dict(k=A + 21 * MB + 1), 3), (dict(p=A + 3), 3), (dict(m=A + 2), 3), (dict(out=A + 64), 4),
    (dict(out=A + 20 * MB), 4), (dict(out=A + 21 * MB), 4), (dict(out=A + 22 * MB), 4), (dict(out=A + 23 * MB), 4),
    (dict(n=0, logits=None, out=None), 0),
]


def _sample_fields(kw):
    f = dict(logits=A, s0=2000, s1=500, dtype=0, n=3, nodes=4, vocab=500, t=A + 20 * MB, k=A + 21 * MB, p=A + 22 * MB,
             m=A + 23 * MB, u=A + 24 * MB, out=A + 10 * MB)
    f.update(kw)
    return f


@pytest.mark.parametrize("kw,want", SAMPLE_BAD + [(dict(u=None), 1), (dict(u=A + 2), 3), (dict(out=A + 24 * MB), 4)])
def test_sample_arguments(lib, kw, want):
    f = _sample_fields(kw)
    assert lib.qnre_sample(*[f[k] for k in ("logits", "s0", "dtype", "n", "vocab", "t", "k", "p", "m", "u", "out")], None) == want


@pytest.mark.parametrize("kw,want", SAMPLE_BAD + [(dict(nodes=0), 1), (dict(nodes=65), 5), (dict(s1=-1), 1), (dict(s1=1 << 41), 5)])
def test_filter_arguments(lib, kw, want):
    f = _sample_fields(kw)
    assert lib.qnre_filter_probs(*[f[k] for k in ("logits", "s0", "s1", "dtype", "n", "nodes", "vocab", "t", "k", "p", "m", "out")],
                                 None) == want


@pytest.mark.parametrize("kw,want", CACHE_BAD)
def test_prefix_calls_check_the_cache(lib, kw, want):
    c = cache(**kw)
    assert lib.qnre_cache_shared_prefix(ctypes.byref(c), A + 200 * MB, 2, A + 201 * MB, 1, A + 202 * MB, None) == want
    assert attention(lib, c=c) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), 1), (dict(g=-1), 1), (dict(g=1025), 5), (dict(n=1025), 5), (dict(rows=None), 1), (dict(groups=None), 1),
    (dict(shared=None), 1), (dict(rows=A + 200 * MB + 2), 3), (dict(groups=A + 201 * MB + 1), 3), (dict(shared=A + 202 * MB + 2), 3),
    (dict(shared=A + 200 * MB), 4), (dict(shared=A + 201 * MB), 4), (dict(shared=A + 128 * MB), 4), (dict(shared=A + 64), 4),
    (dict(g=0, rows=None, groups=None, shared=None), 0),
])
def test_shared_prefix_arguments(lib, kw, want):
    f = dict(rows=A + 200 * MB, n=4, groups=A + 201 * MB, g=2, shared=A + 202 * MB)
    f.update(kw)
    assert lib.qnre_cache_shared_prefix(ctypes.byref(cache()), f["rows"], f["n"], f["groups"], f["g"], f["shared"], None) == want


def attention(lib, **kw):
    f = dict(q=view(A + 200 * MB, [2, 4, 8, 128]), c=cache(), layer=0, rows=A + 210 * MB, groups=A + 211 * MB, g=1,
             shared=A + 212 * MB, mask=None, depths=None, counts=None, scale=0.1, cap=0.0, slopes=None, out=A + 220 * MB,
             lse=A + 230 * MB, ws=A + 240 * MB, size=1 << 32)
    f.update(kw)
    return lib.qnre_prefix_attention(ctypes.byref(f["q"]) if f["q"] else None, ctypes.byref(f["c"]),
                                     *[f[k] for k in ("layer", "rows", "groups", "g", "shared", "mask", "depths", "counts",
                                                      "scale", "cap", "slopes", "out", "lse", "ws", "size")], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(q=view(A + 200 * MB, [2, 4, 7, 128])), 1), (dict(q=view(A + 200 * MB, [2, 4, 8, 64])), 1),
    (dict(q=view(A + 200 * MB, [2, 4, 8, 128], dtype=1)), 1), (dict(q=view(A + 200 * MB, [2, 65, 8, 128])), 5),
    (dict(q=view(A + 200 * MB, [1025, 1, 8, 128])), 5), (dict(q=view(A + 200 * MB + 8, [2, 4, 8, 128])), 3),
    (dict(q=view(A + 200 * MB, [2, 1, 258, 128])), 2),
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(scale=0.0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(cap=-1.0), 1),
    (dict(cap=NAN), 1), (dict(cap=INF), 1), (dict(cap=1e-31), 2), (dict(cap=1e-20, scale=1e30), 2), (dict(g=-1), 1), (dict(g=1025), 5), (dict(groups=None), 1), (dict(shared=None), 1),
    (dict(rows=None), 1), (dict(rows=A + 2), 3), (dict(groups=A + 211 * MB + 2), 3), (dict(shared=A + 212 * MB + 1), 3),
    (dict(mask=A + 213 * MB + 4), 3), (dict(depths=A + 213 * MB + 2), 3), (dict(counts=A + 213 * MB + 2), 3),
    (dict(slopes=A + 213 * MB + 2), 3), (dict(out=None), 1), (dict(out=A + 220 * MB + 8), 3), (dict(ws=None), 1),
    (dict(size=1000), 5), (dict(out=A + 200 * MB), 4), (dict(out=A), 4), (dict(lse=A + 64 * MB), 4), (dict(lse=A + 220 * MB + 16), 4),
    (dict(ws=A + 219 * MB), 4), (dict(lse=A + 212 * MB), 4), (dict(lse=A + 211 * MB + 4), 4), (dict(slopes=A + 230 * MB), 4),
    (dict(mask=A + 230 * MB), 4), (dict(depths=A + 220 * MB), 4),
    (dict(q=view(A + 200 * MB, [0, 4, 8, 128]), rows=None, groups=None, shared=None, out=None, ws=None), 0),
    (dict(q=view(A + 200 * MB, [2, 0, 8, 128]), rows=None, out=None, ws=None), 0),
])
def test_prefix_attention_arguments(lib, kw, want):
    assert attention(lib, **kw) == want


@pytest.mark.parametrize("name", ["out", "lse", "ws"])
@pytest.mark.parametrize("at", [128, 129, 131])
def test_prefix_attention_keeps_off_the_cache_state(lib, name, at):
    c = cache(rows=4, max_blocks=4)
    if name == "ws":  # (it would reach the query otherwise)
        c = cache(block_table=A + 300 * MB, seq_lens=A + 301 * MB, status=A + 303 * MB)
        at += 172
    assert attention(lib, c=c, **{name: A + at * MB}) == 4


def test_prefix_workspace(lib):
    def need(*a):
        n = ctypes.c_uint64()
        return lib.qnre_prefix_attention_workspace_bytes(*a, ctypes.byref(n)), n.value

    assert lib.qnre_prefix_attention_workspace_bytes(1, 1, 8, 8, 64, 0, None) == 1
    for args, want in (((-1, 1, 8, 8, 64, 0), 1), ((1, -1, 8, 8, 64, 0), 1), ((1, 1, 9, 8, 64, 0), 1), ((1, 1, 8, 0, 64, 0), 1),
                       ((1, 1, 8, 8, 96, 0), 2), ((1, 1, 258, 2, 64, 0), 2), ((1025, 1, 8, 8, 64, 0), 5), ((1, 65, 8, 8, 64, 0), 5),
                       ((1, 1, 8, 8, 64, -1), 1)):
        assert need(*args)[0] == want
    # a place of its own for every row's part of either kind, of D floats and a word of four; without groups the words alone
    rows = 128 * 3 * 64
    assert need(128, 3, 64, 8, 128, 5)[1] - need(128, 3, 64, 8, 128, 0)[1] == rows * (2 * 512 + 16) + 128 * 8 * 12
    assert need(0, 1, 8, 8, 128, 1)[0] == 0


class _Call:
    """Calls of the binding on CPU tensors with one argument replaced."""

    def __init__(self, torch):
        z = torch.zeros
        bf, i32 = torch.bfloat16, torch.int32
        pool = z((1, 4, 2, 8, 64), dtype=bf)
        self.cache = qb.PagedCache(pool, torch.zeros_like(pool), z((3, 2), dtype=i32), z(3, dtype=i32), z(4, dtype=i32))
        self.good = dict(q=z((2, 3, 4, 64), dtype=bf), rows=z(2, dtype=i32), groups=z(2, dtype=i32), shared=z(1, dtype=i32),
                         mask=z((2, 3), dtype=torch.int64), out=z((2, 3, 4, 64), dtype=bf), lse=z((2, 3, 4)),
                         counts=z(2, dtype=i32), depths=z((2, 3), dtype=i32), slopes=z(4), ws=z(16, dtype=torch.uint8), cap=1.0,
                         logits=z((2, 50)), trees=z((2, 3, 50), dtype=bf), u=z(2), tokens=z(2, dtype=i32), probs=z((2, 3, 50)),
                         t=z(2), k=z(2, dtype=i32), p=z(2), m=z(2))

    def run(self, i, name, value):
        a, s = dict(self.good, **{name: value}), _Stream()
        try:
            if i == 0:
                qb.qnre_prefix_attention(a["q"], self.cache, 0, a["rows"], a["groups"], a["shared"], a["mask"], a["out"],
                                         lse=a["lse"], counts=a["counts"], depths=a["depths"], softcap=a["cap"],
                                         slopes=a["slopes"], workspace=a["ws"], stream=s)
            elif i == 1:
                qb.qnre_cache_shared_prefix(self.cache, a["rows"], a["groups"], a["shared"], stream=s)
            elif i == 2:
                qb.qnre_sample(a["logits"], a["u"], a["tokens"], a["t"], a["k"], a["p"], a["m"], stream=s)
            else:
                qb.qnre_filter_probs(a["trees"], a["probs"], a["t"], a["k"], a["p"], a["m"], stream=s)
        except Exception as e:
            return type(e).__name__, str(e)
        return "accepted"


def test_native_calls_refuse_as_the_python_ones(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("tensors of the CPU are refused where there is a GPU")
    if qb._native is None:
        pytest.skip("_marshal is not built")
    call = _Call(torch)
    z, i32 = torch.zeros, torch.int32
    wrong = [("ws", z(16, dtype=torch.uint8)), ("ws", None), ("cap", -1.0), ("groups", None), ("shared", None),
             ("groups", z(3, dtype=i32)), ("groups", z(2)), ("shared", z(1)), ("rows", z(3, dtype=i32)), ("mask", z((2, 3), dtype=i32)),
             ("depths", z((3, 2), dtype=i32)), ("depths", z((2, 3))), ("slopes", z(3)), ("slopes", z(4).double()),
             ("counts", z((1, 2), dtype=i32)), ("lse", z((2, 3))), ("out", z((2, 3, 4, 64))), ("q", z((2, 3, 4, 64))),
             ("q", z((2, 3, 4, 64), dtype=torch.bfloat16).transpose(2, 3)), ("logits", z((2, 50)).double()), ("logits", z(2, 50, 1)),
             ("logits", z((50, 2)).t()), ("logits", z((2, 50)).int()), ("u", z(3)), ("u", z(2).half()), ("tokens", z(2)),
             ("tokens", z((2, 1), dtype=i32)), ("t", z(3)), ("t", z(2, dtype=i32)), ("k", z(2)), ("p", z(1)), ("m", z(4)[::2]),
             ("trees", z((2, 50))), ("trees", z((2, 50, 3)).transpose(1, 2)), ("probs", z((2, 3, 50)).half()),
             ("probs", z((2, 3, 51)))]
    native = [call.run(i, *w) for w in wrong for i in range(4)]
    monkeypatch.setattr(qb, "_native", None)
    python = [call.run(i, *w) for w in wrong for i in range(4)]
    assert native == python
    assert sum(x != "accepted" for x in native) >= len(wrong)


def test_rope_table_reads(lib):
    torch = pytest.importorskip("torch")
    for t, kw in ((torch.zeros(8), {}), (torch.zeros((8, 64), dtype=torch.float16), {}), (torch.zeros((64, 8)).t(), {}),
                  (torch.zeros((8, 64)), dict(scaling="ntk")), (torch.zeros((8, 20)), {})):
        with pytest.raises(qb.QnreError):
            qb.qnre_rope_table(t, stream=_Stream(), **kw)
