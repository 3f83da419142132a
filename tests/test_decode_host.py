"""Refusals of the speculative-decoding calls: status codes before anything reaches a GPU."""
import ctypes
import os

import pytest

from ulysses_qkv_proj_gb300 import binding as qb

A = 1 << 32  # addresses that are only ever checked, 16-byte aligned and far apart
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qb.LIB_PATH):
        from ulysses_qkv_proj_gb300 import build
        build.build()
    return qb.load_library()


def cache(**kw):
    f = dict(k=A, v=A + 64 * MB, block_table=A + 128 * MB, seq_lens=A + 129 * MB, page_refs=A + 130 * MB,
             status=A + 131 * MB, scratch=A + 132 * MB, layers=2, pages=4, heads=2, page_size=16, head_dim=128, rows=4,
             max_blocks=4, dtype=0)
    f.update(kw)
    return qb._Cache(*[f[n] for n, _ in qb._Cache._fields_])


def view(ptr, shape, stride=None, dtype=0):
    t = qb._Tensor4()
    t.data = ptr
    if stride is None:
        stride, n = [0] * 4, 1
        for i in reversed(range(4)):
            stride[i], n = n, n * max(1, shape[i])
    for i in range(4):
        t.shape[i], t.stride[i] = shape[i], stride[i]
    t.dtype = dtype
    return t


CACHE_BAD = [
    (dict(k=None), 1), (dict(scratch=None), 1), (dict(pages=0), 1), (dict(max_blocks=0), 1), (dict(rows=-1), 1),
    (dict(head_dim=96), 2), (dict(dtype=2), 2), (dict(page_size=12), 2), (dict(k=A + 8), 3),
    (dict(page_refs=A + 130 * MB + 4), 3), (dict(seq_lens=A + 129 * MB + 2), 3),
    (dict(layers=1 << 16, pages=1 << 16), 5), (dict(rows=1 << 20, max_blocks=1 << 12), 5),
    (dict(max_blocks=1 << 28), 5),
]


@pytest.mark.parametrize("kw,want", CACHE_BAD)
def test_cache_checks(lib, kw, want):
    c = ctypes.byref(cache(**kw))
    L = A + 256 * MB
    assert lib.qnre_cache_truncate(c, L, L + MB, 1, None) == want
    assert lib.qnre_cache_fork(c, L, L + MB, 1, None) == want
    assert lib.qnre_cache_reserve(c, L, L + MB, 1, None) == want
    assert lib.qnre_cache_copy_pages(c, L, L + MB, 1, None) == want
    assert lib.qnre_cache_compact(c, L, L + MB, L + 2 * MB, 1, 4, None) == want


def test_cache_call_arguments(lib):
    c, L = ctypes.byref(cache()), A + 256 * MB
    assert lib.qnre_cache_truncate(None, L, L + MB, 1, None) == 1
    assert lib.qnre_cache_truncate(c, None, L, 1, None) == 1
    assert lib.qnre_cache_truncate(c, L + 2, L, 1, None) == 3
    assert lib.qnre_cache_truncate(c, L, L + MB, -1, None) == 1
    assert lib.qnre_cache_truncate(c, L, L + MB, 1025, None) == 5
    assert lib.qnre_cache_compact(c, L, L + MB, L + 2 * MB, 1, 0, None) == 1
    assert lib.qnre_cache_compact(c, L, L + MB, L + 2 * MB, 1, 65, None) == 5
    for call in (lib.qnre_cache_truncate, lib.qnre_cache_fork, lib.qnre_cache_reserve, lib.qnre_cache_copy_pages):
        assert call(c, None, None, 0, None) == 0


def norm_args(**kw):
    f = dict(q=view(A, [1, 4, 4, 128]), k=view(A + MB, [1, 4, 2, 128]), wq=A + 2 * MB, wk=A + 2 * MB + 256,
             cs=A + 3 * MB, n_pos=8, rot=128, style=0, pos=None, qo=view(A + 4 * MB, [1, 4, 4, 128]),
             ko=view(A + 5 * MB, [1, 4, 2, 128]))
    f.update(kw)
    return f


NORM_BAD = [
    (dict(q=view(None, [1, 4, 4, 128])), 1),
    (dict(q=view(A, [1, 4, 4, 96])), 2),
    (dict(q=view(A, [1, 4, 4, 128], dtype=2)), 2),
    (dict(q=view(A + 8, [1, 4, 4, 128])), 3),
    (dict(q=view(A, [1, 4, 4, 128], [2048, 516, 128, 1])), 3),
    (dict(q=view(A, [1, 4, 4, 128], [2048, 1, 512, 4])), 3),
    (dict(q=view(A, [1, 3, 4, 128])), 1),
    (dict(k=view(A + MB, [1, 4, 2, 128], dtype=1)), 1),
    (dict(k=view(A + MB, [1, 4, 2, 64])), 1),
    (dict(wq=None), 1), (dict(wk=A + 8), 3), (dict(cs=None), 1), (dict(cs=A + 4), 3), (dict(n_pos=0), 1),
    (dict(rot=130), 1), (dict(rot=0), 1), (dict(rot=24), 1), (dict(style=2), 1), (dict(pos=A + 6 * MB + 2), 3),
]


@pytest.mark.parametrize("kw,want", NORM_BAD)
def test_norm_checks(lib, kw, want):
    a = norm_args(**kw)
    head = [ctypes.byref(a["q"]), ctypes.byref(a["k"]), a["wq"], a["wk"], a["cs"], a["n_pos"], a["rot"], a["style"], a["pos"]]
    assert lib.qnre_qk_norm_rope(*head, ctypes.byref(a["qo"]), ctypes.byref(a["ko"]), None) == want
    g = view(A + 8 * MB, [1, 4, 4, 128]), view(A + 9 * MB, [1, 4, 2, 128])
    assert lib.qnre_qk_norm_rope_backward(ctypes.byref(g[0]), ctypes.byref(g[1]), *head, ctypes.byref(a["qo"]),
                                          ctypes.byref(a["ko"]), A + 10 * MB, A + 10 * MB + 512, A + 11 * MB, 1 << 24,
                                          None) == want
    v = view(A + 12 * MB, [1, 4, 2, 128])
    c = cache(k=A + 200 * MB, v=A + 264 * MB)
    assert lib.qnre_qkv_norm_rope_append(head[0], head[1], ctypes.byref(v), *head[2:], ctypes.byref(a["qo"]),
                                         ctypes.byref(c), 0, A + 13 * MB, None, None) == want


def test_norm_aliases(lib):
    def run(**kw):
        a = norm_args(**kw)
        return lib.qnre_qk_norm_rope(ctypes.byref(a["q"]), ctypes.byref(a["k"]), a["wq"], a["wk"], a["cs"], a["n_pos"],
                                     a["rot"], a["style"], a["pos"], ctypes.byref(a["qo"]), ctypes.byref(a["ko"]), None)
    assert run(qo=view(A + 256, [1, 4, 4, 128])) == 4                     # over its own input, shifted
    assert run(qo=view(A + MB, [1, 4, 4, 128])) == 4                      # over the other input
    assert run(qo=view(A + 4 * MB, [1, 4, 4, 128]), ko=view(A + 4 * MB + 1024, [1, 4, 2, 128])) == 4
    assert run(qo=view(A + 4 * MB, [1, 4, 4, 128], [512, 128, 128, 1])) == 1  # writes an element twice
    # head bands of one buffer: overlapping spans, no shared element
    s = [4 * 768, 768, 128, 1]
    ok = dict(q=view(A, [0, 4, 4, 128], s), k=view(A + 1024, [0, 4, 2, 128], s), qo=view(A, [0, 4, 4, 128], s),
              ko=view(A + 1024, [0, 4, 2, 128], s))
    assert run(**ok) == 0
    s = [4 * 768, 768, 128, 1]
    bad = dict(q=view(A, [1, 4, 4, 128], s), k=view(A + 1024 - 256, [1, 4, 2, 128], s), qo=view(A, [1, 4, 4, 128], s),
               ko=view(A + 5 * MB, [1, 4, 2, 128]))
    assert run(**bad) == 4


def test_norm_backward_and_append_arguments(lib):
    a = norm_args()
    head = [ctypes.byref(a["q"]), ctypes.byref(a["k"]), a["wq"], a["wk"], a["cs"], 8, 128, 0, None]
    g = view(A + 8 * MB, [1, 4, 4, 128]), view(A + 9 * MB, [1, 4, 2, 128])

    def back(gq=g[0], dq=a["qo"], dw=A + 10 * MB, ws=A + 11 * MB, n=1 << 24):
        return lib.qnre_qk_norm_rope_backward(ctypes.byref(gq), ctypes.byref(g[1]), *head, ctypes.byref(dq),
                                              ctypes.byref(a["ko"]), dw, A + 10 * MB + 512, ws, n, None)
    assert back(gq=view(A + 8 * MB, [1, 4, 3, 128])) == 1
    assert back(dq=view(A, [1, 4, 4, 128])) == 4
    assert back(dw=None) == 1
    assert back(dw=A + 10 * MB + 2) == 3
    assert back(dw=A + 10 * MB + 512) == 4
    assert back(ws=None) == 1
    assert back(ws=A + 11 * MB + 4) == 3
    assert back(n=64) == 5
    v = view(A + 12 * MB, [1, 4, 2, 128])

    def append(c=None, v=v, layer=0, rows=A + 13 * MB):
        c = c or cache(k=A + 200 * MB, v=A + 264 * MB)
        return lib.qnre_qkv_norm_rope_append(head[0], head[1], ctypes.byref(v), *head[2:], ctypes.byref(a["qo"]),
                                             ctypes.byref(c), layer, rows, None, None)
    assert append(v=view(A + 12 * MB, [1, 4, 3, 128])) == 1
    assert append(layer=2) == 1
    assert append(layer=-1) == 1
    assert append(rows=None) == 1
    assert append(rows=A + 13 * MB + 1) == 3
    assert append(c=cache(heads=3)) == 1
    assert append(c=cache(dtype=1)) == 1
    assert append(c=cache(k=A)) == 4
    n = ctypes.c_uint64()
    assert lib.qnre_qk_norm_rope_workspace_bytes(96, ctypes.byref(n)) == 2
    assert lib.qnre_qk_norm_rope_workspace_bytes(128, None) == 1


def test_binding_checks_types_and_shapes():
    torch = pytest.importorskip("torch")
    k = torch.zeros((1, 2, 1, 8, 64), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(qb.QnreError):
        qb.PagedCache(k[0], k[0], i(1, 1), i(1), i(2))
    with pytest.raises(qb.QnreError):
        qb.PagedCache(k, k.half(), i(1, 1), i(1), i(2))
    with pytest.raises(qb.QnreError):
        qb.PagedCache(k, k.clone(), i(1, 1), i(2), i(2))
    with pytest.raises(qb.QnreError):
        qb.PagedCache(k, k.clone(), i(1, 1).long(), i(1), i(2))
    with pytest.raises(qb.QnreError):
        qb._i32("x", i(3), 4)


def attention(lib, **kw):
    f = dict(q=view(A + 200 * MB, [2, 4, 8, 128]), c=cache(), layer=0, rows=A + 210 * MB, mask=None, counts=None,
             scale=0.1, out=A + 220 * MB, lse=A + 230 * MB, ws=A + 240 * MB, size=1 << 30)
    f.update(kw)
    return lib.qnre_tree_attention(ctypes.byref(f["q"]) if f["q"] else None, ctypes.byref(f["c"]), f["layer"], f["rows"],
                                   f["mask"], f["counts"], f["scale"], f["out"], f["lse"], f["ws"], f["size"], None)


@pytest.mark.parametrize("kw,want", CACHE_BAD)
def test_attention_checks_the_cache(lib, kw, want):
    assert attention(lib, c=cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(q=view(A + 200 * MB, [2, 4, 7, 128])), 1), (dict(q=view(A + 200 * MB, [2, 4, 8, 64])), 1),
    (dict(q=view(A + 200 * MB, [2, 4, 8, 128], dtype=1)), 1), (dict(q=view(A + 200 * MB, [2, 65, 8, 128])), 5),
    (dict(q=view(A + 200 * MB, [1025, 1, 8, 128])), 5), (dict(q=view(A + 200 * MB + 8, [2, 4, 8, 128])), 3),
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(rows=None), 1), (dict(rows=A + 2), 3), (dict(mask=A + 210 * MB + 4), 3),
    (dict(counts=A + 210 * MB + 2), 3), (dict(out=None), 1), (dict(out=A + 220 * MB + 8), 3), (dict(ws=None), 1),
    (dict(size=1000), 5), (dict(out=A + 200 * MB), 4), (dict(out=A), 4), (dict(lse=A + 64 * MB), 4),
    (dict(lse=A + 220 * MB + 16), 4), (dict(ws=A + 219 * MB), 4), (dict(q=view(A + 200 * MB, [0, 4, 8, 128]), rows=None), 0),
])
def test_attention_arguments(lib, kw, want):
    assert attention(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), 1), (dict(nodes=0), 1), (dict(vocab=0), 1), (dict(nodes=65), 5), (dict(vocab=1 << 31), 5),
    (dict(p=None), 1), (dict(tokens=None), 1), (dict(u=None), 1), (dict(path=None), 1), (dict(nxt=None), 1),
    (dict(ps0=-1), 1), (dict(qs1=1 << 41), 5), (dict(p=A + 2), 3), (dict(path=A + 40 * MB + 1), 3),
    (dict(path=A + 64), 4), (dict(kept=A + 30 * MB), 4), (dict(nxt=A + 50 * MB), 4), (dict(n=0, p=None), 0),
])
def test_verify_arguments(lib, kw, want):
    f = dict(p=A, ps0=4000, ps1=1000, q=A + 10 * MB, qs0=4000, qs1=1000, n=3, nodes=4, vocab=1000, tokens=A + 20 * MB,
             parents=A + 30 * MB, node_counts=None, u=A + 35 * MB, s=A + 36 * MB, path=A + 40 * MB, kept=A + 50 * MB,
             nxt=A + 60 * MB)
    f.update(kw)
    assert lib.qnre_verify_tree(*[f[k] for k in ("p", "ps0", "ps1", "q", "qs0", "qs1", "n", "nodes", "vocab", "tokens",
                                                 "parents", "node_counts", "u", "s", "path", "kept", "nxt")], None) == want


def test_tree_mask_arguments(lib):
    f = lib.qnre_tree_masks
    assert f(None, 1, 4, A, A + MB, None) == 1
    assert f(A, -1, 4, None, None, None) == 1
    assert f(A, 1, 0, None, None, None) == 1
    assert f(A, 1, 65, None, None, None) == 5
    assert f(A + 2, 1, 4, None, None, None) == 3
    assert f(A, 1, 4, A + MB + 4, None, None) == 3
    assert f(A, 1, 4, A + 8, None, None) == 4
    assert f(A, 1, 4, A + MB, A + MB, None) == 4
    assert f(None, 0, 4, None, None, None) == 0
    n = ctypes.c_uint64()
    assert lib.qnre_tree_attention_workspace_bytes(96, ctypes.byref(n)) == 2
    assert lib.qnre_tree_attention_workspace_bytes(64, None) == 1


def test_native_reads_agree_with_python_ones(lib, monkeypatch):
    """_marshal gives what the Python reads give, and lets them name what is wrong."""
    torch = pytest.importorskip("torch")
    native = qb._native
    if native is None:
        pytest.skip("_marshal is not built")
    base = torch.zeros((3, 4, 10, 64), dtype=torch.float16)
    views = [base, base[:, :, 2:7], base.transpose(0, 1), base.to(torch.bfloat16)[1:, ::2], base.float(), base[:0]]
    ints = [torch.zeros(5, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32).t(),
            torch.zeros(5, dtype=torch.int64), torch.zeros(5)]

    def all_of():
        r = []
        for v in views + [base[0], base.double(), base.int()]:
            try:
                r.append(qb._view4(v))
            except qb.QnreError as e:
                r.append(str(e))
        for t in ints:
            for read in (lambda t, *s: qb._i32("x", t, *s), lambda t, *s: qb._f32("x", t, *s), lambda t, *s: qb._i64("x", t, *s)):
                for shape in ((5,), (2, 3), (3, 2)):
                    try:
                        r.append(read(t, *shape))
                    except qb.QnreError as e:
                        r.append(str(e))
        for w, like in ((base[0, 0, 0], base), (base[0, 0, 0], base.float()), (base[0, 0, :, 0], base), (base[0, 0, 0, :32], base)):
            try:
                r.append(qb._weight("x", w, 64, like))
            except qb.QnreError as e:
                r.append(str(e))
        return r

    views = [v for v in views]
    with_native = all_of()
    assert [tuple(qb._sizes(v)) for v in views] == [tuple(v.shape) for v in views]
    monkeypatch.setattr(qb, "_native", None)
    without = all_of()
    # base.float() makes a new tensor each time only in the list above, so addresses agree
    assert with_native == without
    assert any(isinstance(x, str) for x in without) and any(isinstance(x, bytes) for x in without)


class _Stream:
    cuda_stream = 0


def test_whole_native_calls_refuse_as_the_python_ones(lib, monkeypatch):
    """A norm, its gradient and an append with one argument wrong at a time: the same error with and without _marshal."""
    torch = pytest.importorskip("torch")
    if qb._native is None:
        pytest.skip("_marshal is not built")
    bf = torch.bfloat16
    good = dict(q=torch.zeros((2, 3, 4, 64), dtype=bf), k=torch.zeros((2, 3, 2, 64), dtype=bf),
                v=torch.zeros((2, 3, 2, 64), dtype=bf), wq=torch.ones(64, dtype=bf), wk=torch.ones(64, dtype=bf),
                table=torch.zeros((8, 32)), pos=torch.zeros((2, 3), dtype=torch.int32),
                qo=torch.zeros((2, 3, 4, 64), dtype=bf), ko=torch.zeros((2, 3, 2, 64), dtype=bf),
                gq=torch.zeros((2, 3, 4, 64), dtype=bf), gk=torch.zeros((2, 3, 2, 64), dtype=bf),
                dwq=torch.zeros(64), dwk=torch.zeros(64), ws=torch.zeros(1 << 20, dtype=torch.uint8),
                rows=torch.zeros(2, dtype=torch.int32), counts=None, layer=0, style="rotate_half")
    pool = torch.zeros((1, 4, 2, 8, 64), dtype=bf)
    cache = qb.PagedCache(pool, torch.zeros_like(pool), torch.zeros((3, 2), dtype=torch.int32),
                          torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    s = _Stream()
    calls = [
        lambda a: qb.qnre_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"], a["qo"], a["ko"],
                                       rope_style=a["style"], stream=s),
        lambda a: qb.qnre_qk_norm_rope_backward(a["gq"], a["gk"], a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"],
                                                a["qo"], a["ko"], a["dwq"], a["dwk"], a["ws"], rope_style=a["style"],
                                                stream=s),
        lambda a: qb.qnre_qkv_norm_rope_append(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["table"], a["pos"], a["qo"], cache,
                                               a["layer"], a["rows"], a["counts"], rope_style=a["style"], stream=s),
    ]
    wrong = [("style", "none"), ("layer", 5), ("layer", -1), ("rows", torch.zeros(3, dtype=torch.int32)),
             ("rows", torch.zeros(2, dtype=torch.int64)), ("counts", torch.zeros((2, 1), dtype=torch.int32)),
             ("ws", torch.zeros(16, dtype=torch.uint8)), ("ws", torch.zeros((1 << 11, 1 << 10), dtype=torch.uint8).t())]
    for name in ("q", "k", "v", "qo", "ko", "gq", "gk"):
        t = good[name]
        wrong += [(name, t[0]), (name, t.float()), (name, t.half()), (name, t.to_sparse()), (name, t[..., :32]),
                  (name, t.transpose(2, 3)), (name, t.double())]
    for name in ("wq", "wk", "dwq", "dwk"):
        t = good[name]
        wrong += [(name, t[:32]), (name, t.half()), (name, t[None]), (name, torch.zeros((64, 2), dtype=t.dtype)[:, 0])]
    wrong += [("table", good["table"][0]), ("table", good["table"].t()), ("table", good["table"].double()),
              ("table", torch.zeros((8, 24))), ("pos", good["pos"].long()), ("pos", good["pos"][:1]), ("pos", good["pos"].t())]

    def outcomes():
        r = []
        for name, value in wrong:
            for i, call in enumerate(calls):
                # (an argument that the call has, so that a launch is never reached)
                if name in ((("v", "rows", "counts", "layer", "gq", "gk", "dwq", "dwk", "ws")),
                            ("v", "rows", "counts", "layer"), ("ko", "gq", "gk", "dwq", "dwk", "ws"))[i]:
                    continue
                try:
                    call({**good, name: value})
                    r.append((name, i, None))
                except Exception as e:  # the Python reads of a sparse tensor raise torch's own errors
                    r.append((name, i, type(e).__name__, str(e)))
        return r

    with_native = outcomes()
    assert all(len(x) == 4 for x in with_native)
    monkeypatch.setattr(qb, "_native", None)
    assert with_native == outcomes()


def test_whole_native_cache_and_tree_calls_refuse_as_the_python_ones(lib, monkeypatch):
    """The same of the cache's bookkeeping, the attention and the verification."""
    torch = pytest.importorskip("torch")
    if qb._native is None:
        pytest.skip("_marshal is not built")
    bf, i32 = torch.bfloat16, torch.int32
    pool = torch.zeros((1, 4, 2, 8, 64), dtype=bf)
    cache = qb.PagedCache(pool, torch.zeros_like(pool), torch.zeros((3, 2), dtype=i32), torch.zeros(3, dtype=i32),
                          torch.zeros(4, dtype=i32))
    s = _Stream()
    rows = [torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros((2, 1), dtype=i32),
            torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=i32)[::2], torch.zeros(2), torch.zeros(2, dtype=i32).to_sparse(),
            torch.zeros(1025, dtype=i32)]
    path = [torch.zeros((2, 3), dtype=i32), torch.zeros((2, 65), dtype=i32), torch.zeros(2, dtype=i32),
            torch.zeros((3, 2), dtype=i32).t(), torch.zeros((2, 0), dtype=i32), torch.zeros((2, 3))]
    good = dict(q=torch.zeros((2, 3, 4, 64), dtype=bf), rows=rows[0], mask=torch.zeros((2, 3), dtype=torch.int64),
                out=torch.zeros((2, 3, 4, 64), dtype=bf), lse=torch.zeros((2, 3, 4)), counts=rows[0], scale=0.125, layer=0,
                ws=torch.zeros(64 << 20, dtype=torch.uint8))
    probs = dict(target=torch.rand((2, 3, 50)), draft=torch.rand((2, 3, 50)), tokens=torch.zeros((2, 3), dtype=i32),
                 parents=torch.zeros((2, 3), dtype=i32), accept=torch.zeros((2, 3)), sample=torch.zeros(2),
                 path=torch.zeros((2, 3), dtype=i32), counts=torch.zeros(2, dtype=i32), next=torch.zeros(2, dtype=i32),
                 nodes=None)
    att_wrong = [("q", good["q"][0]), ("q", good["q"].half()), ("q", good["q"][:, :, :3]), ("q", good["q"].to_sparse()),
                 ("rows", rows[1]), ("rows", rows[3]), ("mask", good["mask"].int()), ("mask", good["mask"][:1]),
                 ("mask", good["mask"].t()), ("out", good["out"].half()), ("out", good["out"][:, :2]),
                 ("out", good["out"].transpose(0, 1)), ("lse", good["lse"].double()), ("lse", good["lse"][0]),
                 ("counts", rows[1]), ("scale", -1.0), ("scale", float("nan")), ("scale", 0), ("scale", float("inf")),
                 ("layer", 1), ("layer", -1), ("ws", None), ("ws", good["ws"][:64]), ("ws", good["ws"][::2])]
    ver_wrong = [("target", probs["target"][0]), ("target", probs["target"].double()), ("target", probs["target"].transpose(1, 2)),
                 ("target", probs["target"].to_sparse()), ("draft", probs["draft"][:, :2]), ("draft", probs["draft"].half()),
                 ("tokens", probs["tokens"].long()), ("parents", probs["parents"][:1]), ("accept", probs["accept"].double()),
                 ("sample", probs["sample"][:1]), ("path", probs["path"].t()), ("counts", torch.zeros(2)),
                 ("next", torch.zeros(3, dtype=i32)), ("nodes", torch.zeros(3, dtype=i32)), ("tokens", probs["path"]),
                 ("next", probs["counts"])]

    def outcomes():
        r = []

        def note(call):
            try:
                call()
                r.append(None)
            except Exception as e:
                r.append((type(e).__name__, str(e)))

        for bad in rows[1:]:
            for two in (lambda a, b: qb.qnre_cache_truncate(cache, a, b, s), lambda a, b: qb.qnre_cache_fork(cache, a, b, s),
                        lambda a, b: qb.qnre_cache_reserve(cache, a, b, s),
                        lambda a, b: qb.qnre_cache_copy_pages(cache, a, b, s)):
                note(lambda: two(bad, rows[0]))
                note(lambda: two(rows[0], bad))
            note(lambda: qb.qnre_cache_compact(cache, bad, path[0], rows[0], s))
            note(lambda: qb.qnre_cache_compact(cache, rows[0], path[0], bad, s))
        for bad in path[1:]:
            note(lambda: qb.qnre_cache_compact(cache, rows[0], bad, rows[0], s))
        for name, value in att_wrong:
            a = {**good, name: value}
            note(lambda: qb.qnre_tree_attention(a["q"], cache, a["layer"], a["rows"], a["mask"], a["out"], a["lse"],
                                                a["counts"], a["scale"], a["ws"], s))
        for name, value in ver_wrong:
            a = {**probs, name: value}
            note(lambda: qb.qnre_verify_tree(a["target"], a["draft"], a["tokens"], a["parents"], a["accept"], a["sample"],
                                             a["path"], a["counts"], a["next"], a["nodes"], s))
        return r

    with_native = outcomes()
    assert None not in with_native
    monkeypatch.setattr(qb, "_native", None)
    assert with_native == outcomes()


def _calls(torch, cache, dev="cpu"):
    """Every decoding call as (name, arguments by name, call of them); all of them would be accepted on one device."""
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, device=dev)
    norm = dict(q=z(2, 3, 4, 64), k=z(2, 3, 2, 64), wq=z(64), wk=z(64), table=z(8, 32, dtype=torch.float32),
                pos=z(2, 3, dtype=i32))
    outs = dict(qo=z(2, 3, 4, 64), ko=z(2, 3, 2, 64))
    rows = dict(a=z(2, dtype=i32), b=z(2, dtype=i32))
    s = _Stream()
    r = [("norm", {**norm, **outs}, lambda a: qb.qnre_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"], a["qo"],
                                                                   a["ko"], stream=s)),
         ("backward", {**norm, **outs, "gq": z(2, 3, 4, 64), "gk": z(2, 3, 2, 64), "dwq": z(64, dtype=torch.float32),
                       "dwk": z(64, dtype=torch.float32), "ws": z(1 << 20, dtype=torch.uint8)},
          lambda a: qb.qnre_qk_norm_rope_backward(a["gq"], a["gk"], a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"], a["qo"],
                                                  a["ko"], a["dwq"], a["dwk"], a["ws"], stream=s)),
         ("append", {**norm, "v": z(2, 3, 2, 64), "qo": outs["qo"], "rows": rows["a"], "counts": rows["b"]},
          lambda a: qb.qnre_qkv_norm_rope_append(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["table"], a["pos"], a["qo"], cache, 0,
                                                 a["rows"], a["counts"], stream=s)),
         ("compact", {**rows, "path": z(2, 3, dtype=i32)},
          lambda a: qb.qnre_cache_compact(cache, a["a"], a["path"], a["b"], s)),
         ("masks", dict(parents=z(2, 3, dtype=i32), masks=z(2, 3, dtype=torch.int64), depths=z(2, 3, dtype=i32)),
          lambda a: qb.qnre_tree_masks(a["parents"], a["masks"], a["depths"], s)),
         ("attention", dict(q=z(2, 3, 4, 64), rows=rows["a"], mask=z(2, 3, dtype=torch.int64), out=z(2, 3, 4, 64),
                            lse=z(2, 3, 4, dtype=torch.float32), counts=rows["b"], ws=z(64 << 20, dtype=torch.uint8)),
          lambda a: qb.qnre_tree_attention(a["q"], cache, 0, a["rows"], a["mask"], a["out"], a["lse"], a["counts"], None, a["ws"], s)),
         ("verify", dict(target=z(2, 3, 50, dtype=torch.float32), draft=z(2, 3, 50, dtype=torch.float32), tokens=z(2, 3, dtype=i32),
                         parents=z(2, 3, dtype=i32), accept=z(2, 3, dtype=torch.float32), sample=z(2, dtype=torch.float32),
                         path=z(2, 3, dtype=i32), counts=z(2, dtype=i32), next=z(2, dtype=i32), nodes=z(2, dtype=i32)),
          lambda a: qb.qnre_verify_tree(a["target"], a["draft"], a["tokens"], a["parents"], a["accept"], a["sample"], a["path"],
                                        a["counts"], a["next"], a["nodes"], s))]
    for name in ("truncate", "fork", "reserve", "copy_pages"):
        call = getattr(qb, "qnre_cache_" + name)
        r.append((name, rows, lambda a, call=call: call(cache, a["a"], a["b"], s)))
    return r


class _Entries:
    """Stands in for the library: every entry point answers 0 and notes that it was reached."""

    def __init__(self):
        self.reached = []

    def __getattr__(self, name):
        return lambda *a: self.reached.append(name) or 0


@pytest.mark.parametrize("native", [True, False])
def test_tensors_of_another_device_are_refused(lib, monkeypatch, native):
    """One argument at a time on another device (meta), then all on the CPU of a machine that has CUDA."""
    torch = pytest.importorskip("torch")
    if native and qb._native is None:
        pytest.skip("_marshal is not built")
    pool = lambda dev: [torch.zeros((1, 4, 2, 8, 64), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    i = lambda dev, *s: torch.zeros(s, dtype=torch.int32, device=dev)
    cache = qb.PagedCache(*pool("cpu"), i("cpu", 3, 2), i("cpu", 3), i("cpu", 4))
    for at in range(5):
        dev = ["cpu"] * 5
        dev[at] = "meta"
        k, v = pool(dev[0])[0], pool(dev[1])[1]
        with pytest.raises(qb.QnreError, match="one device"):
            qb.PagedCache(k, v, i(dev[2], 3, 2), i(dev[3], 3), i(dev[4], 4))
    if not native:
        monkeypatch.setattr(qb, "_native", None)
    fake = _Entries()
    monkeypatch.setattr(qb, "load_library", lambda *a: fake)
    for name, args, call in _calls(torch, cache):
        for key in args:
            with pytest.raises(qb.QnreError, match="current CUDA device"):
                call({**args, key: args[key].to("meta")})
    assert not fake.reached
    # a machine with CUDA: the same tensors, all on the CPU, do not reach an entry point either (the native reads ask
    # torch's library itself, so only the Python ones can be told that there is one)
    if not native:
        for name, args, call in _calls(torch, cache):
            call(args)
        assert len(fake.reached) == 11
        monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
        for name, args, call in _calls(torch, cache):
            with pytest.raises(qb.QnreError, match="current CUDA device"):
                call(args)
        assert len(fake.reached) == 11


def test_the_build_goes_on_without_the_native_reads(monkeypatch, tmp_path, capsys):
    """g++ that fails on torch's headers: printed, no older module left, nothing raised."""
    pytest.importorskip("torch")
    import types
    from ulysses_qkv_proj_gb300 import build
    old = tmp_path / "_marshal.so"
    old.write_bytes(b"older")
    monkeypatch.setattr(build, "MARSHAL_PATH", str(old))
    monkeypatch.setattr(build.shutil, "which", lambda name: "/usr/bin/" + name)
    monkeypatch.setattr(build.os.path, "exists", lambda p, real=os.path.exists: p.endswith("Python.h") or real(p))
    monkeypatch.setattr(build.subprocess, "run",
                        lambda *a, **k: types.SimpleNamespace(returncode=1, stdout="", stderr="no such header"))
    assert build.build_marshal() == ""
    assert not old.exists() and "no such header" in capsys.readouterr().err
