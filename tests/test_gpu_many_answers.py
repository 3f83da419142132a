"""The operators for many answers from one prompt together, as a server runs them; and what each call must hold besides its results."""
import os
import sys

import numpy as np
import pytest
import torch

import _decode as D
from test_gpu_prefix_attention import Case
from test_gpu_sample import settings, token, weights
from test_gpu_speculative_example import _logits

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _qb():
    from ulysses_qkv_proj_gb300 import binding as qb
    return qb


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prompts_and_samples(check=True):
    """Two prompts, forked into three and four samples, five steps each: table, append, search for common pages, attention,
    sampling, filtered probabilities, compaction.  Checked against 64 bits; all that was written, as bytes."""
    qb = _qb()
    gen = torch.Generator(device="cuda").manual_seed(5)
    Hq, Hk, dim, V, ps, cap = 4, 2, 64, 501, 16, 20.0
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    cache = qb.alloc_paged_cache(1, 80, Hk, ps, dim, 9, 8)
    cache.k.zero_(), cache.v.zero_()
    table = torch.empty((128, 48), device="cuda")          # three quarters of a head turn
    qb.qnre_rope_table(table, theta=1e5, scaling="yarn", factor=2.0, original=64.0)
    w = [1 + 0.1 * randn(dim) for _ in range(2)]
    head = randn(Hq * dim, V)
    lens, S = [70, 45], 70
    keys, values = [], []

    def append(x, rows, counts, pos):
        n, s = x.shape[:2]
        q_out = torch.zeros((n, s, Hq, dim), dtype=x.dtype, device="cuda")
        qb.qnre_qkv_norm_rope_append(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:], *w, table, None, q_out, cache, 0, rows, counts)
        k = D.norm_rope(x[:, :, Hq:Hq + Hk].cpu(), w[1].cpu(), table.cpu(), pos, "rotate_half").bfloat16()
        return q_out, k, x[:, :, Hq + Hk:].cpu()

    x = randn(2, S, Hq + 2 * Hk, dim)
    prompts = _i32([7, 8])
    qb.qnre_cache_reserve(cache, prompts, _i32(lens))
    _, k, v = append(x, prompts, _i32(lens), torch.arange(S).expand(2, S))
    # (an append of more than 64 tokens is kept in two parts)
    qb.qnre_cache_compact(cache, prompts, torch.arange(40, device="cuda").int().expand(2, 40).contiguous(), _i32([40, 40]))
    qb.qnre_cache_reserve(cache, prompts, _i32([30, 5]))
    append(x[:, 40:], prompts, _i32([30, 5]), torch.arange(40, S).expand(2, S - 40))
    qb.qnre_cache_compact(cache, prompts, torch.arange(30, device="cuda").int().expand(2, 30).contiguous(), _i32([30, 5]))
    members, rows = [0, 0, 0, 1, 1, 1, 1], [4, 0, 6, 1, 3, 2, 5]
    qb.qnre_cache_fork(cache, _i32([7 + p for p in members]), _i32(rows))
    for p in members:
        keys.append(k[p, :lens[p]])
        values.append(v[p, :lens[p]])
    d_rows, groups, shared = _i32(rows), _i32([0, 3, 7]), _i32([-1, -1])
    n = len(rows)
    s = settings(n, T=[0.7, 0.0, 1.0, 0.9, 1.2, 0.8, 1.0], k=[0, 0, 20, 0, 5, 0, 0], p=[1.0, 1.0, 0.9, 0.8, 1.0, 0.95, 1.0],
                 m=[0.0, 0.0, 0.0, 0.0, 0.0, 0.05, 0.1])
    wrote = [table]
    out = torch.zeros((n, 1, Hq, dim), dtype=torch.bfloat16, device="cuda")
    lse, probs = torch.zeros((n, 1, Hq), device="cuda"), torch.zeros((n, 1, V), device="cuda")
    tokens = _i32([0] * n)
    for step in range(5):
        x = randn(n, 1, Hq + 2 * Hk, dim)
        qb.qnre_cache_reserve(cache, d_rows, _i32([1] * n))
        pos = torch.tensor([[len(t)] for t in keys])
        q, k, v = append(x, d_rows, None, pos)
        qb.qnre_cache_shared_prefix(cache, d_rows, groups, shared)
        qb.qnre_prefix_attention(q, cache, 0, d_rows, groups, shared, None, out, lse=lse, softcap=cap,
                                 workspace=qb.prefix_attention_workspace(q, cache))
        logits = out.view(n, -1).float() @ head.float()
        u = torch.rand(n, generator=gen, device="cuda")
        qb.qnre_sample(logits, u, tokens, **s)
        qb.qnre_filter_probs(logits[:, None], probs, **s)
        qb.qnre_cache_compact(cache, d_rows, _i32([[0]] * n), _i32([1] * n))
        wrote += [t.clone() for t in (q, out, lse, logits, tokens, probs, shared)]
        keys = [torch.cat([a, k[i]]) for i, a in enumerate(keys)]
        values = [torch.cat([a, v[i]]) for i, a in enumerate(values)]
        if not check:
            continue
        assert shared.tolist() == [70 // ps * ps, 45 // ps * ps]
        for i in range(n):
            z = logits[i].cpu().numpy()
            kept = weights(z, *(float(s[a][i]) if a != "top_k" else int(s[a][i]) for a in ("temperature", "top_k", "top_p", "min_p")))
            assert int(tokens[i]) == token(kept, float(u[i]))
            assert ((probs[i, 0].cpu().numpy() > 0) == (kept > 0)).all()
            for h in range(Hq):
                # K lies in the cache rounded once more than the reference here: half a bf16 step of every product
                sc = keys[i][:, h // 2].double() @ q[i, 0, h].cpu().double() * dim ** -0.5
                loose = float((keys[i][:, h // 2].double().abs() @ q[i, 0, h].cpu().double().abs()).max()) * dim ** -0.5 * 2.0 ** -8
                p = torch.softmax(cap * torch.tanh(sc / cap), 0)
                ref = p @ values[i][:, h // 2].double()
                size = p @ values[i][:, h // 2].double().abs()
                err = (out[i, 0, h].cpu().double() - ref).abs()
                assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * loose) * size).all()
    assert cache.status() == 0
    held = cache.block_table.cpu()
    assert cache.page_refs.cpu().tolist() == [int((held == p).sum()) for p in range(80)]
    wrote += [cache.k, cache.v, cache.block_table, cache.seq_lens, cache.page_refs]
    return [t.contiguous().view(torch.uint8).cpu() for t in wrote]


def test_samples_of_prompts():
    _prompts_and_samples()


def test_python_reads_give_the_native_ones_bits(monkeypatch):
    qb = _qb()
    qb.load_library()
    if qb._native is None:
        pytest.skip("_marshal is not built")
    native = _prompts_and_samples(check=False)
    monkeypatch.setattr(qb, "_native", None)
    assert all(torch.equal(a, b) for a, b in zip(native, _prompts_and_samples(check=False)))


def test_tensors_of_the_host_are_refused():
    qb = _qb()
    c = Case([(3, 64)], [9], Hq=4, Hk=2, seed=1)
    q = c.prepare()
    x, u, t = torch.zeros((2, 9), device="cuda"), torch.zeros(2, device="cuda"), _i32([0, 0])
    good = dict(rows=c.d_rows, groups=c.d_groups, shared=c.d_shared, out=c.out, lse=c.lse, ws=c.ws)

    def attend(**kw):
        a = dict(good, **kw)
        qb.qnre_prefix_attention(q, c.cache, 1, a["rows"], a["groups"], a["shared"], None, a["out"], lse=a["lse"], workspace=a["ws"])

    attend()
    for name, value in good.items():
        with pytest.raises(qb.QnreError):
            attend(**{name: value.cpu()})
    for name in ("rows", "groups", "shared"):
        with pytest.raises(qb.QnreError):
            a = dict(good, **{name: good[name].cpu()})
            qb.qnre_cache_shared_prefix(c.cache, a["rows"], a["groups"], a["shared"])
    with pytest.raises(qb.QnreError):
        attend(ws=c.ws[:1000])
    with pytest.raises(qb.QnreError):
        attend(ws=c.ws[8:])
    for args in ((x.cpu(), u, t), (x, u.cpu(), t), (x, u, t.cpu())):
        with pytest.raises(qb.QnreError):
            qb.qnre_sample(*args)
    with pytest.raises(qb.QnreError):
        qb.qnre_sample(x, u, t, temperature=torch.ones(2))
    with pytest.raises(qb.QnreError):
        qb.qnre_filter_probs(x[:, None], torch.zeros((2, 1, 9)))
    with pytest.raises(qb.QnreError):
        qb.qnre_rope_table(torch.zeros((4, 64)))
    assert not t.any()


def test_caches_of_more_than_two_billion_elements():
    """Pages beyond 2^31 elements: attention, a missing value's own part, and the search."""
    qb = _qb()
    c = Case([(4, 256)], [130, 3], Hq=8, Hk=2, page=128, dim=128, layers=1, layer=0, seed=2)
    c.values[1][c.common[1] + 1, 0, 5] = float("inf")
    c.fill()
    pages = 2 ** 31 // (2 * 128 * 128) + 200
    low = c.k.shape[1]
    shift = pages - low
    pools = []
    for small in (c.k, c.v):
        pool = torch.empty((1, pages, 2, 128, 128), dtype=c.dt, device="cuda")
        pool[0, shift:] = small[0].cuda()
        pools.append(pool)
    table = torch.where(c.table >= 0, c.table + shift, c.table)
    q = c.prepare()
    c.cache = qb.PagedCache(*pools, table.cuda(), c.seq.cuda(), torch.ones(pages, dtype=torch.int32, device="cuda"))
    c.d_shared.fill_(-1)
    qb.qnre_cache_shared_prefix(c.cache, c.d_rows, c.d_groups, c.d_shared)
    assert c.d_shared.tolist() == [256]
    c.call(q)
    assert (c.out[1, 0, :4, 5] == float("inf")).all()
    c.check(c.out.cpu(), c.lse.cpu(), only=[0, 2, 3])


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import parallel_sampling
    return parallel_sampling


def test_example_follows_the_model(ex):
    """Greedy samples of a prompt are alike, and each token is the 64-bit model's best, up to what bf16 layers blur."""
    model = ex.device_table(ex.Model(sharpness=30.0), scaling="linear", factor=2.0)
    prompts = torch.randint(0, model.vocab, (2, 90), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    texts = ex.sample(model, prompts, 3, 10, settings=dict(temperature=torch.zeros(6, device="cuda")))
    for prompt, group in zip(prompts, texts):
        assert (group == group[0]).all()
        z = _logits(model, torch.cat([prompt, group[0]]))
        for i, t in enumerate(group[0].tolist()):
            row = z[len(prompt) - 1 + i]
            assert row.max() - row[t] <= 0.05 * row.std()


def test_example_keeps_the_cache_whole(ex):
    model = ex.Model()
    prompts = torch.randint(0, model.vocab, (3, 37), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    s = ex.Sampler(model, prompts, 4, max_tokens=100, settings=dict(temperature=torch.full((12,), 1.2, device="cuda")))
    gen = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(20):
        t = s.step(gen)
        assert ((t >= 0) & (t < model.vocab)).all()
    c = s.cache
    assert c.status() == 0 and s.shared.tolist() == [32] * 3
    assert c.seq_lens.cpu().tolist() == [56] * 12 + [36] * 3
    held = c.block_table.cpu()
    assert c.page_refs.cpu().tolist() == [int((held == p).sum()) for p in range(c.k.shape[1])]
