"""Every decoding call as the binding makes it without its native module: accepted, with the same bits."""
import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu


def _step():
    """One serving step from prompt to compaction and a norm with its gradient; all that the calls wrote, as bytes."""
    from ulysses_qkv_proj_gb300 import binding as qb
    gen = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    n, Hq, Hk, dim, V = 2, 8, 2, 64, 1000
    cache = qb.alloc_paged_cache(1, 24, Hk, 16, dim, 4, 6)
    cache.k.zero_(), cache.v.zero_()
    rows, w = i32([2, 0]), [1 + 0.1 * randn(dim) for _ in range(2)]
    cs = D.angles(128, dim).cuda()
    wrote = []
    parents = i32([[-1, 0, 0, 1], [-1, 0, 1, 2]])
    masks, depths = torch.zeros((n, 4), dtype=torch.int64, device="cuda"), i32([[0] * 4] * n)
    qb.qnre_tree_masks(parents, masks, depths)
    for S, chain in ((40, True), (4, False)):
        x = randn(n, S, Hq + 2 * Hk, dim)
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
        out, att = (torch.zeros((n, S, Hq, dim), dtype=x.dtype, device="cuda") for _ in range(2))
        lse = torch.zeros((n, S, Hq), device="cuda")
        counts = None if chain else i32([4, 3])
        pos = None if chain else (cache.seq_lens[rows.long()][:, None] + depths).contiguous()
        qb.qnre_cache_reserve(cache, rows, i32([S] * n))
        qb.qnre_qkv_norm_rope_append(q, k, v, *w, cs, pos, out, cache, 0, rows, counts)
        qb.qnre_tree_attention(out, cache, 0, rows, None if chain else masks, att, lse=lse, counts=counts,
                               scale=None if chain else 0.11, workspace=qb.tree_attention_workspace(out, cache))
        wrote += [out, att, lse]
        if chain:
            qb.qnre_cache_compact(cache, rows, torch.arange(S, device="cuda").int().expand(n, S).contiguous(), i32([S] * n))
            qb.qnre_cache_fork(cache, i32([2]), i32([1]))
    p, d = (torch.rand((n, 4, V + 2), generator=gen, device="cuda")[:, :, 1:1 + V] for _ in range(2))
    path, kept, following = i32([[9] * 4] * n), i32([9] * n), i32([9] * n)
    for draft in (d / d.sum(-1, keepdim=True), None):
        qb.qnre_verify_tree(p / p.sum(-1, keepdim=True), draft, i32([[0, 5, 6, 7]] * n), parents,
                            torch.rand((n, 4), generator=gen, device="cuda"), torch.rand(n, generator=gen, device="cuda"), path,
                            kept, following, node_counts=i32([4, 3]))
        wrote += [path.clone(), kept.clone(), following.clone()]
    qb.qnre_cache_compact(cache, rows, path, kept)
    qb.qnre_cache_truncate(cache, i32([1]), i32([17]))
    qb.qnre_cache_copy_pages(cache, i32([0]), i32([20]))
    x, g = randn(2, 9, Hq + Hk, dim), randn(2, 9, Hq + Hk, dim)
    y = torch.zeros_like(x)
    qb.qnre_qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:], *w, cs, None, y[:, :, :Hq], y[:, :, Hq:], rope_style="interleaved")
    dx, dw = torch.zeros_like(x), [torch.zeros(dim, device="cuda") for _ in range(2)]
    qb.qnre_qk_norm_rope_backward(g[:, :, :Hq], g[:, :, Hq:], x[:, :, :Hq], x[:, :, Hq:], *w, cs, None, dx[:, :, :Hq],
                                  dx[:, :, Hq:], *dw, qb.qk_norm_rope_workspace(x), rope_style="interleaved")
    assert cache.status() == 0
    wrote += [cache.k, cache.v, cache.block_table, cache.seq_lens, cache.page_refs, masks, depths, y, dx, *dw]
    return [t.contiguous().view(torch.uint8).cpu() for t in wrote]


def test_python_reads_give_the_native_ones_bits(monkeypatch):
    from ulysses_qkv_proj_gb300 import binding as qb
    qb.load_library()
    if qb._native is None:
        pytest.skip("_marshal is not built")
    native = _step()
    assert all(t.any() for t in native)
    monkeypatch.setattr(qb, "_native", None)
    assert all(torch.equal(a, b) for a, b in zip(native, _step()))
