"""Several answers from each prompt on one GPU, end to end.

    python examples/parallel_sampling.py

The model of speculative_decode.py, its rotary table made on the device
(qnre_rope_table).  Each prompt enters the paged cache once and is forked into
its samples (qnre_cache_fork); every step finds the pages that the samples
share (qnre_cache_shared_prefix), lets them attend to the prompt together
(qnre_prefix_attention) and draws each sample's next token from its logits with the
sample's own settings (qnre_sample).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from speculative_decode import Decoder, Model, qb  # noqa: E402


class Sampler(Decoder):
    """`samples` rows for each prompt, side by side; the prompts' own rows behind them."""

    def __init__(self, model, prompts, samples, max_tokens=1024, page_size=16, settings=None):
        n, self.samples = prompts.shape[0], samples
        super().__init__(model, n * (samples + 1), max_tokens, page_size)
        everyone = self.rows
        self.rows = everyone[n * samples:].contiguous()
        self.prefill(prompts)
        source, self.rows = self.rows, everyone[:n * samples].contiguous()
        qb.qnre_cache_fork(self.cache, source.repeat_interleave(samples).contiguous(), self.rows)
        self.last = prompts[:, -1].repeat_interleave(samples).contiguous()
        self.groups = torch.arange(n + 1, dtype=torch.int32, device="cuda") * samples
        self.shared = torch.empty(n, dtype=torch.int32, device="cuda")
        self.settings = settings or {}
        self.root = torch.zeros((n * samples, 1), dtype=torch.int32, device="cuda")

    def forward(self, tokens, parents):
        """Logits of the prompts' next tokens (parents None: a chain), or of one token of each sample, which reads its
        prompt together with the others."""
        m, cache = self.m, self.cache
        n, nodes = tokens.shape
        qb.qnre_cache_reserve(cache, self.rows, self.full(nodes))
        q, out = (torch.empty((n, nodes, m.heads, qb.HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if parents is None:
            workspace = qb.tree_attention_workspace(q, cache)
        else:
            qb.qnre_cache_shared_prefix(cache, self.rows, self.groups, self.shared)
            workspace = qb.prefix_attention_workspace(q, cache)
        x = m.embed[tokens.long()]
        raw = qb.alloc_outputs(self.plan, n, nodes)
        for layer in range(m.layers):
            qw, kw = m.norms[layer]
            qb.qnre_forward(self.plan, x[None], m.w_qkv[layer], qw, kw, m.cos_sin, None, raw)
            qb.qnre_qkv_norm_rope_append(raw["q"][0], raw["k"][0], raw["v"][0], qw, kw, m.cos_sin, None, q, cache, layer,
                                         self.rows)
            if parents is None:
                qb.qnre_tree_attention(q, cache, layer, self.rows, None, out, workspace=workspace)
            else:
                qb.qnre_prefix_attention(q, cache, layer, self.rows, self.groups, self.shared, None, out, workspace=workspace)
            x = x + out.view(n, nodes, -1) @ m.w_out[layer]
        return (x @ m.head).float()

    def step(self, generator):
        """The next token of every sample."""
        logits = self.forward(self.last[:, None], self.root)
        u = torch.rand(self.rows.numel(), generator=generator, device="cuda")
        following = torch.empty_like(self.rows)
        qb.qnre_sample(logits[:, 0], u, following, **self.settings)
        qb.qnre_cache_compact(self.cache, self.rows, self.root, self.full(1))
        self.last = following
        return following


def sample(model, prompts, samples, new_tokens, seed=0, settings=None):
    """Tokens [prompts, samples, new_tokens]."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = Sampler(model, prompts, samples, max_tokens=prompts.shape[1] + new_tokens, settings=settings)
    texts = torch.stack([s.step(gen) for _ in range(new_tokens)], 1)
    if s.cache.status() != 0:
        raise RuntimeError("the cache reported an error")
    return texts.view(prompts.shape[0], samples, new_tokens)


def device_table(model, **scaling):
    """The model with a rotary table made on the device."""
    model.cos_sin = torch.empty_like(model.cos_sin)
    qb.qnre_rope_table(model.cos_sin, **scaling)
    return model


def main():
    model = device_table(Model(), scaling="yarn", factor=4.0, original=1024.0)
    prompts = torch.randint(0, model.vocab, (3, 150), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    rows = 3 * 8
    fp = lambda x: torch.full((rows,), x, device="cuda")
    texts = sample(model, prompts, 8, 30, settings=dict(temperature=fp(0.8), top_k=fp(50).int(), top_p=fp(0.95)))
    different = sum(len({tuple(t) for t in group}) for group in texts.tolist())
    print(f"{rows} samples of 3 prompts, 30 tokens each: {different} different texts")


if __name__ == "__main__":
    main()
