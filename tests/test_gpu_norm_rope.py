"""qnre_qk_norm_rope, its gradient and its cache form against 64-bit plain forms.

Tolerances: one rounding to the output type (half a step of the value) plus the
fp32 chain, at most some 16 roundings (2^-20) of the sizes that enter a channel
forward; the gradient's means of up to 128 products add 128 * 2^-24 = 2^-17."""
import math

import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


def _inputs(B, S, Hq, Hk, dim, dt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    proj = torch.randn((B, S, Hq + 2 * Hk, dim), generator=gen).to(dt)
    w = [(1 + 0.1 * torch.randn(dim, generator=gen)).to(dt) for _ in range(2)]
    return proj, w[0], w[1], gen


def _close(got, ref, tol, what):
    got = got.double().cpu()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN pattern differs"
    over = ((got - ref).abs() - tol)[~nan]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: worst excess {over.max():.3g}"


def _fwd_tol(ref, x, w, cs, style, dt):
    return D.half_step(dt) * ref.abs() * 1.01 + 2.0 ** -19 * D.pair_size(x, w, cs, style) + 2.0 ** -25


CASES = [  # B, S, Hq, Hk, dim, rot, style, dtype
    (1, 1, 1, 1, 128, 128, "rotate_half", "bf16"),
    (2, 7, 8, 2, 128, 128, "interleaved", "fp16"),
    (3, 33, 7, 7, 64, 64, "rotate_half", "fp16"),
    (1, 129, 56, 14, 128, 64, "rotate_half", "bf16"),
    (2, 50, 5, 3, 64, 16, "interleaved", "bf16"),
    (1, 40, 9, 1, 64, 48, "rotate_half", "bf16"),
    (1, 3000, 64, 8, 128, 128, "rotate_half", "bf16"),
    (1, 17, 33, 5, 128, 112, "interleaved", "fp16"),
]


@pytest.mark.parametrize("B,S,Hq,Hk,dim,rot,style,dtype", CASES)
def test_forward(B, S, Hq, Hk, dim, rot, style, dtype):
    qb, dt = _qb(), DT[dtype]
    proj, qw, kw, gen = _inputs(B, S, Hq, Hk, dim, dt)
    cs = D.angles(S + 5, rot)
    pos = torch.randint(0, S + 5, (B, S), generator=gen, dtype=torch.int32)
    pos[0, 0] = S + 5 if S > 1 else 0       # outside the table
    if S > 2:
        pos[0, 2] = -1
    d = proj.cuda()
    out = torch.full((B, S, Hq + Hk, dim), 7.0, dtype=dt, device="cuda")
    qb.qnre_qk_norm_rope(d[:, :, :Hq], d[:, :, Hq:Hq + Hk], qw.cuda(), kw.cuda(), cs.cuda(), pos.cuda(),
                         out[:, :, :Hq], out[:, :, Hq:], rope_style=style)
    for got, x, w in ((out[:, :, :Hq], proj[:, :, :Hq], qw), (out[:, :, Hq:], proj[:, :, Hq:Hq + Hk], kw)):
        ref = D.norm_rope(x, w, cs, pos, style)
        _close(got, ref, _fwd_tol(ref, x, w, cs, style, dt), "forward")


def test_in_place_strided_and_default_positions():
    """In place on one projection buffer whose sequences are the faster axis; V is left alone."""
    qb, dt = _qb(), torch.bfloat16
    B, S, Hq, Hk, dim = 3, 20, 6, 2, 128
    proj, qw, kw, _ = _inputs(B, S, Hq, Hk, dim, dt, 3)
    cs = D.angles(S, dim)
    buf = proj.transpose(0, 1).contiguous().cuda()       # [S, B, heads, dim]
    view = buf.transpose(0, 1)
    q, k = view[:, :, :Hq], view[:, :, Hq:Hq + Hk]
    qb.qnre_qk_norm_rope(q, k, qw.cuda(), kw.cuda(), cs.cuda(), None, q, k)
    pos = torch.arange(S).expand(B, S)
    for got, x, w in ((q, proj[:, :, :Hq], qw), (k, proj[:, :, Hq:Hq + Hk], kw)):
        ref = D.norm_rope(x, w, cs, pos, "rotate_half")
        _close(got, ref, _fwd_tol(ref, x, w, cs, "rotate_half", dt), "in place")
    assert torch.equal(view[:, :, Hq + Hk:].cpu(), proj[:, :, Hq + Hk:])


def test_zero_rows_and_large_values():
    qb, dt = _qb(), torch.bfloat16
    x = torch.zeros((1, 3, 2, 64), dtype=dt)
    x[0, 1] = 1e18
    x[0, 2] = 1e-20
    w = torch.ones(64, dtype=dt)
    cs = D.angles(3, 64)
    out = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    qb.qnre_qk_norm_rope(x.cuda(), x.cuda(), w.cuda(), w.cuda(), cs.cuda(), None, *out)
    ref = D.norm_rope(x, w, cs, torch.arange(3)[None], "rotate_half")
    for got in out:
        _close(got, ref, _fwd_tol(ref, x, w, cs, "rotate_half", dt), "extremes")
        assert not got[0, 0].any()


@pytest.mark.parametrize("B,S,Hq,Hk,dim,rot,style,dtype", CASES)
def test_gradient(B, S, Hq, Hk, dim, rot, style, dtype):
    qb, dt = _qb(), DT[dtype]
    proj, qw, kw, gen = _inputs(B, S, Hq, Hk, dim, dt, 1)
    g = torch.randn((B, S, Hq + Hk, dim), generator=gen).to(dt)
    cs = D.angles(S + 2, rot)
    pos = torch.randint(0, S + 2, (B, S), generator=gen, dtype=torch.int32)
    d, gd = proj.cuda(), g.cuda()
    gq, gk = gd[:, :, :Hq], gd[:, :, Hq:]
    dw = [torch.full((dim,), 9.0, device="cuda") for _ in range(2)]
    ws = qb.qk_norm_rope_workspace(d)
    # in place: the gradient of the outputs becomes that of the inputs
    qb.qnre_qk_norm_rope_backward(gq, gk, d[:, :, :Hq], d[:, :, Hq:Hq + Hk], qw.cuda(), kw.cuda(), cs.cuda(),
                                  pos.cuda(), gq, gk, *dw, ws, rope_style=style)
    for got, gw, gx, x, w in ((gq, dw[0], g[:, :, :Hq], proj[:, :, :Hq], qw),
                              (gk, dw[1], g[:, :, Hq:], proj[:, :, Hq:Hq + Hk], kw)):
        dx, dwr, size, wsize = D.norm_rope_grad(gx, x, w, cs, pos, style)
        _close(got, dx, D.half_step(dt) * dx.abs() * 1.01 + 2.0 ** -16 * size + 2.0 ** -25, "dx")
        # at most 256 additions in a row before the pairwise levels
        _close(gw, dwr, 2.0 ** -16 * wsize + 1e-30, "dw")


def test_gradient_against_differences():
    """Directional derivatives of the 64-bit forward by central differences."""
    qb, dt = _qb(), torch.float16
    B, S, Hq, Hk, dim, style = 1, 9, 3, 1, 64, "interleaved"
    proj, qw, kw, gen = _inputs(B, S, Hq, Hk, dim, dt, 5)
    g = torch.randn((B, S, Hq + Hk, dim), generator=gen).to(dt)
    cs, pos = D.angles(S, 32), torch.arange(S)[None]
    dq = torch.empty((B, S, Hq, dim), dtype=dt, device="cuda")
    dk = torch.empty((B, S, Hk, dim), dtype=dt, device="cuda")
    dw = [torch.empty(dim, device="cuda") for _ in range(2)]
    gd, d = g.cuda(), proj.cuda()
    qb.qnre_qk_norm_rope_backward(gd[:, :, :Hq], gd[:, :, Hq:], d[:, :, :Hq], d[:, :, Hq:Hq + Hk], qw.cuda(),
                                  kw.cuda(), cs.cuda(), None, dq, dk, *dw, qb.qk_norm_rope_workspace(d),
                                  rope_style=style)
    for got, gw, gx, x, w in ((dq, dw[0], g[:, :, :Hq], proj[:, :, :Hq], qw),
                              (dk, dw[1], g[:, :, Hq:], proj[:, :, Hq:Hq + Hk], kw)):
        x, w, gx = x.double(), w.double(), gx.double()
        _, _, size, wsize = D.norm_rope_grad(gx, x, w, cs, pos, style)
        for _ in range(4):
            vx = torch.randn(x.shape, generator=gen, dtype=torch.float64)
            vw = torch.randn(w.shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            diff = ((D.norm_rope(x + h * vx, w, cs, pos, style) - D.norm_rope(x - h * vx, w, cs, pos, style)) * gx).sum() / (2 * h)
            dgot = got.double().cpu()
            tol = ((D.half_step(dt) * dgot.abs() * 1.02 + 2.0 ** -16 * size + 2.0 ** -25) * vx.abs()).sum() + 1e-6
            assert abs((dgot * vx).sum() - diff) <= tol
            diff = ((D.norm_rope(x, w + h * vw, cs, pos, style) - D.norm_rope(x, w - h * vw, cs, pos, style)) * gx).sum() / (2 * h)
            assert abs((gw.double().cpu() * vw).sum() - diff) <= (2.0 ** -16 * wsize * vw.abs()).sum() + 1e-6


def test_gradient_repeats_bit_for_bit_and_empty_batch():
    qb, dt = _qb(), torch.bfloat16
    proj, qw, kw, gen = _inputs(2, 400, 8, 2, 128, dt, 2)
    g = torch.randn((2, 400, 10, 128), generator=gen).to(dt).cuda()
    d, cs = proj.cuda(), D.angles(400, 128).cuda()
    runs = []
    for _ in range(2):
        dq, dk = torch.empty_like(d[:, :, :8]), torch.empty_like(d[:, :, :2])
        dw = [torch.empty(128, device="cuda") for _ in range(2)]
        qb.qnre_qk_norm_rope_backward(g[:, :, :8], g[:, :, 8:], d[:, :, :8], d[:, :, 8:10], qw.cuda(), kw.cuda(), cs,
                                      None, dq, dk, *dw, qb.qk_norm_rope_workspace(d))
        runs.append([dq, dk, *dw])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    dw = [torch.ones(128, device="cuda") for _ in range(2)]
    e, ek = d[:0, :, :8], d[:0, :, 8:10]
    qb.qnre_qk_norm_rope_backward(g[:0, :, :8], g[:0, :, 8:], e, ek, qw.cuda(), kw.cuda(), cs, None,
                                  torch.empty_like(e), torch.empty_like(ek), *dw, qb.qk_norm_rope_workspace(d))
    assert not dw[0].any() and not dw[1].any()


@pytest.mark.parametrize("page,dim,dtype,counts", [(16, 128, "bf16", None), (48, 64, "fp16", [3, 0, 5, 9]),
                                                   (8, 128, "fp16", None)])
def test_append(page, dim, dtype, counts):
    """K and V land in the rows' slots, crossing pages; q_out is the plain forward; nothing else changes."""
    qb, dt = _qb(), DT[dtype]
    n, S, Hq, Hk, layers = 4, 5, 6, 2, 2
    proj, qw, kw, gen = _inputs(n, S, Hq, Hk, dim, dt, 4)
    lens = [0, page - 2, 3 * page, 37]
    rows_total, blocks = 6, 2 + 3 * page // page + -(-40 // page)
    pages = rows_total * blocks
    perm = torch.randperm(pages, generator=gen).int().view(rows_total, blocks)
    pools = [torch.randn((layers, pages, Hk, page, dim), generator=gen).to(dt) for _ in range(2)]
    rows = torch.tensor([5, 0, 3, 2], dtype=torch.int32)
    seq = torch.zeros(rows_total, dtype=torch.int32)
    seq[rows.long()] = torch.tensor(lens, dtype=torch.int32)
    cache = qb.PagedCache(pools[0].cuda(), pools[1].cuda(), perm.cuda(), seq.cuda(),
                          torch.ones(pages, dtype=torch.int32, device="cuda"))
    cs = D.angles(3 * page + S, dim)
    d = proj.cuda()
    q_out = torch.empty((n, S, Hq, dim), dtype=dt, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32).cuda() if counts else None
    qb.qnre_qkv_norm_rope_append(d[:, :, :Hq], d[:, :, Hq:Hq + Hk], d[:, :, Hq + Hk:], qw.cuda(), kw.cuda(),
                                 cs.cuda(), None, q_out, cache, 1, rows.cuda(), cnt)
    pos = torch.tensor(lens)[:, None] + torch.arange(S)
    ref = D.norm_rope(proj[:, :, :Hq], qw, cs, pos, "rotate_half")
    _close(q_out, ref, _fwd_tol(ref, proj[:, :, :Hq], qw, cs, "rotate_half", dt), "q_out")
    k = proj[:, :, Hq:Hq + Hk]
    kref = D.norm_rope(k, kw, cs, pos, "rotate_half")
    tol = _fwd_tol(kref, k, kw, cs, "rotate_half", dt)
    gk, gv = cache.k.cpu(), cache.v.cpu()
    want = [p.clone() for p in pools]
    for i in range(n):
        for s in range(min(S, counts[i]) if counts else S):
            p, slot = perm[rows[i], (lens[i] + s) // page], (lens[i] + s) % page
            _close(gk[1, p, :, slot], kref[i, s], tol[i, s], "appended k")
            want[0][1, p, :, slot] = gk[1, p, :, slot]
            want[1][1, p, :, slot] = proj[i, s, Hq + Hk:]
    bits = [t.view(torch.int16) for t in (gk, want[0], gv, want[1])]  # positions past a short table are NaN rows
    assert torch.equal(bits[0], bits[1]) and torch.equal(bits[2], bits[3])
    assert cache.status() == 0


def test_append_without_pages_is_reported_and_skipped():
    qb, dt = _qb(), torch.bfloat16
    proj, qw, kw, _ = _inputs(3, 2, 2, 1, 128, dt, 6)
    cache = qb.alloc_paged_cache(1, 4, 1, 8, 128, 2, 2)
    cache.k.zero_(), cache.v.zero_()
    cache.block_table[1, 0] = 4                       # outside the cache
    d, cs = proj.cuda(), D.angles(8, 128).cuda()
    out = torch.empty((3, 2, 2, 128), dtype=dt, device="cuda")
    qb.qnre_qkv_norm_rope_append(d[:, :, :2], d[:, :, 2:3], d[:, :, 3:], qw.cuda(), kw.cuda(), cs, None, out, cache,
                                 0, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
    assert cache.status() == qb.CACHE_BAD_PAGE | qb.CACHE_BAD_ROW
    assert cache.status() == 0
    assert not cache.k.any() and not cache.v.any()


def test_other_stream_and_graph():
    """The calls run on the stream they are given and replay from a graph on new inputs."""
    qb, dt = _qb(), torch.bfloat16
    proj, qw, kw, _ = _inputs(1, 64, 8, 2, 128, dt, 7)
    cs = D.angles(64, 128).cuda()
    d, w = proj.cuda(), (qw.cuda(), kw.cuda())
    out = torch.empty((1, 64, 10, 128), dtype=dt, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qb.qnre_qk_norm_rope(d[:, :, :8], d[:, :, 8:10], *w, cs, None, out[:, :, :8], out[:, :, 8:])
    again, *_ = _inputs(1, 64, 8, 2, 128, dt, 8)
    d.copy_(again)
    g.replay()
    torch.cuda.synchronize()
    ref = D.norm_rope(again[:, :, :8], qw, cs.cpu(), torch.arange(64)[None], "rotate_half")
    _close(out[:, :, :8], ref, _fwd_tol(ref, again[:, :, :8], qw, cs.cpu(), "rotate_half", dt), "graph")


def test_gradient_replays_from_a_graph():
    """A captured gradient gives the eager one's bits on new inputs."""
    qb, dt = _qb(), torch.bfloat16
    proj, qw, kw, gen = _inputs(2, 90, 8, 2, 128, dt, 9)
    g = torch.randn((2, 90, 10, 128), generator=gen).to(dt).cuda()
    d, cs, w = proj.cuda(), D.angles(90, 128).cuda(), (qw.cuda(), kw.cuda())
    ws = qb.qk_norm_rope_workspace(d)

    def run(out):
        qb.qnre_qk_norm_rope_backward(g[:, :, :8], g[:, :, 8:], d[:, :, :8], d[:, :, 8:10], *w, cs, None, *out, ws)

    make = lambda: [torch.empty((2, 90, 8, 128), dtype=dt, device="cuda"), torch.empty((2, 90, 2, 128), dtype=dt, device="cuda"),
                    torch.empty(128, device="cuda"), torch.empty(128, device="cuda")]
    captured, eager = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(captured)
    again, _, _, gen = _inputs(2, 90, 8, 2, 128, dt, 10)
    d.copy_(again)
    g.copy_(torch.randn((2, 90, 10, 128), generator=gen).to(dt))
    graph.replay()
    run(eager)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, eager))


@pytest.mark.parametrize("S,Hq,dim,style,dtype", [(262144, 64, 128, "rotate_half", "bf16"), (1 << 20, 16, 64, "interleaved", "fp16"),
                                                  (3000000, 1, 128, "interleaved", "bf16")])
def test_weight_gradients_of_large_batches(S, Hq, dim, style, dtype):
    """Millions of equal terms, whose sums' roundings all lie on one side.

    Tolerance: a term's own 16 roundings, and one for each addition it passes: 62 and 64 in its thread's lower levels,
    one for each 1024 steps (of one or two terms) of the thread, 32 in the block, 42 among the blocks."""
    qb, dt = _qb(), DT[dtype]
    proj, qw, kw, gen = _inputs(1, 1, 1, 1, dim, dt, 11)
    g = torch.randn((1, 1, 2, dim), generator=gen).to(dt)
    cs, pos = D.angles(8, dim), 5
    x, kx = (proj[:, :, i:i + 1].cuda().expand(1, S, h, dim).contiguous() for i, h in ((0, Hq), (1, 1)))
    gq, gk = (g[:, :, i:i + 1].cuda().expand(1, S, h, dim).contiguous() for i, h in ((0, Hq), (1, 1)))
    dw = [torch.empty(dim, device="cuda") for _ in range(2)]
    qb.qnre_qk_norm_rope_backward(gq, gk, x, kx, qw.cuda(), kw.cuda(), cs.cuda(),
                                  torch.full((1, S), pos, dtype=torch.int32, device="cuda"), gq, gk, *dw,
                                  qb.qk_norm_rope_workspace(x), rope_style=style)
    for got, i, heads, w in ((dw[0], 0, Hq, qw), (dw[1], 1, 1, kw)):
        _, one, _, size = D.norm_rope_grad(g[:, :, i:i + 1], proj[:, :, i:i + 1], w, cs, torch.full((1, 1), pos), style)
        n = S * heads
        adds = 62 + 64 + n / (304 * 8 * 1024) + 32 + 42
        _close(got, n * one, n * (2.0 ** -20 * size + adds * 2.0 ** -24 * one.abs()), "dw")


@pytest.mark.parametrize("B", [1, 3])
def test_head_major_bands_in_place(B):
    """q and k as head bands of one [B, H, S, D] buffer: normalised in place, their gradients in place, and an append."""
    qb, dt = _qb(), torch.bfloat16
    S, Hq, Hk, dim = 20, 6, 2, 128
    proj, qw, kw, gen = _inputs(B, S, Hq, Hk, dim, dt, 12)
    cs, pos = D.angles(S, dim), torch.arange(S).expand(B, S)
    w = qw.cuda(), kw.cuda()

    def bands(x):
        v = x.transpose(1, 2).contiguous().cuda().transpose(1, 2)      # [B, S, H, D] over [B, H, S, D]
        return v, v[:, :, :Hq], v[:, :, Hq:Hq + Hk], v[:, :, Hq + Hk:]

    _, q, k, v = bands(proj)
    qb.qnre_qk_norm_rope(q, k, *w, cs.cuda(), None, q, k)
    for got, x, wt in ((q, proj[:, :, :Hq], qw), (k, proj[:, :, Hq:Hq + Hk], kw)):
        ref = D.norm_rope(x, wt, cs, pos, "rotate_half")
        _close(got, ref, _fwd_tol(ref, x, wt, cs, "rotate_half", dt), "in place")
    assert torch.equal(v.cpu(), proj[:, :, Hq + Hk:])

    g = torch.randn((B, S, Hq + 2 * Hk, dim), generator=gen).to(dt)
    (_, q, k, _), (_, gq, gk, _) = bands(proj), bands(g)
    dw = [torch.empty(dim, device="cuda") for _ in range(2)]
    qb.qnre_qk_norm_rope_backward(gq, gk, q, k, *w, cs.cuda(), None, gq, gk, *dw, qb.qk_norm_rope_workspace(q))
    for got, i, n, wt in ((gq, 0, Hq, qw), (gk, Hq, Hk, kw)):
        dx, _, size, _ = D.norm_rope_grad(g[:, :, i:i + n], proj[:, :, i:i + n], wt, cs, pos, "rotate_half")
        _close(got, dx, D.half_step(dt) * dx.abs() * 1.01 + 2.0 ** -16 * size + 2.0 ** -25, "dx")

    cache = qb.alloc_paged_cache(1, 4 * B, Hk, 8, dim, B, 4)
    rows, room = torch.arange(B, dtype=torch.int32, device="cuda"), torch.full((B,), S, dtype=torch.int32, device="cuda")
    qb.qnre_cache_reserve(cache, rows, room)
    _, q, k, v = bands(proj)
    qb.qnre_qkv_norm_rope_append(q, k, v, *w, cs.cuda(), None, q, cache, 0, rows)
    ref = D.norm_rope(proj[:, :, :Hq], qw, cs, pos, "rotate_half")
    _close(q, ref, _fwd_tol(ref, proj[:, :, :Hq], qw, cs, "rotate_half", dt), "append")
    page = cache.block_table[:, 2].long()
    assert torch.equal(cache.v[0, page, :, 1].cpu(), proj[:, 17, Hq + Hk:]) and cache.status() == 0
