"""examples/speculative_decode.py: the operators run together as a decoder runs them."""
import os
import sys

import pytest
import torch

import _decode as D

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import speculative_decode
    return speculative_decode


def _logits(m, tokens):
    """The model in 64 bits on one whole sequence (values rounded where the model rounds them)."""
    rnd = lambda x: x.bfloat16().double()
    S = len(tokens)
    pos = torch.arange(S)[None]
    x = m.embed[tokens.long()].double()
    later = torch.triu(torch.ones((S, S), dtype=torch.bool, device="cuda"), 1)
    for layer in range(m.layers):
        y = rnd(x @ m.w_qkv[layer].double()).view(S, 3, m.heads, 128)
        q, k = (rnd(D.norm_rope(y[None, :, i].cpu(), m.norms[layer][i].cpu(), m.cos_sin[:S].cpu(), pos, "rotate_half")[0].cuda())
                for i in range(2))
        s = torch.einsum("shd,thd->hst", q, k) * 128 ** -0.5
        p = s.masked_fill(later, float("-inf")).softmax(-1)
        o = rnd(torch.einsum("hst,thd->shd", p, y[:, 2])).reshape(S, -1)
        x = rnd(x + o @ m.w_out[layer].double())
    return x @ m.head.double()


@pytest.mark.parametrize("nodes,branch", [(1, 1), (8, 2), (33, 3)])
def test_greedy_decoding_follows_the_model(ex, nodes, branch):
    """Every greedy token is the 64-bit model's best on the emitted prefix, up to what bf16 layers blur: their
    logits are off by some 0.004 standard deviations, two of them by less than 0.05."""
    model = ex.Model(sharpness=30.0)
    prompts = torch.randint(0, model.vocab, (3, 90), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    texts, steps = ex.generate(model, prompts, 12, nodes=nodes, branch=branch, greedy=True)
    assert steps <= 12
    for prompt, text in zip(prompts, texts):
        seq = torch.cat([prompt, torch.tensor(text, dtype=torch.int32, device="cuda")])
        z = _logits(model, seq)
        for i, token in enumerate(text):
            row = z[len(prompt) - 1 + i]
            assert row.max() - row[token] <= 0.05 * row.std()


def test_sampled_decoding_keeps_the_cache_whole(ex):
    model = ex.Model()
    prompts = torch.randint(0, model.vocab, (5, 20), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    d = ex.Decoder(model, 5, max_tokens=200)
    d.prefill(prompts)
    gen = torch.Generator(device="cuda").manual_seed(0)
    last, total = prompts[:, -1].contiguous(), torch.full((5,), 19)
    for _ in range(12):
        last, emitted = d.step(last, 15, 3, gen)
        assert ((emitted >= 0).sum(1) >= 1).all() and (emitted < model.vocab).all() and (last >= 0).all()
        total += (emitted >= 0).sum(1).cpu()
    # every emitted token but the last one of each row is in the cache, in pages of that row alone
    c = d.cache
    assert c.status() == 0
    assert c.seq_lens.cpu().tolist() == total.tolist()
    held = c.block_table.cpu()
    assert (held >= 0).sum(1).tolist() == [-(-x // 16) for x in total.tolist()]
    ids = held[held >= 0]
    assert len(set(ids.tolist())) == len(ids) and int(c.page_refs.sum()) == len(ids)
    qb = ex.qb
    qb.qnre_cache_truncate(c, d.rows, d.full(0))
    assert not c.page_refs.any() and not c.seq_lens.any()
