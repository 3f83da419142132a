"""Speculative decoding on one GPU with the library's own kernels, end to end.

    python examples/speculative_decode.py

A small random transformer of attention layers: the fused projection
(qnre_forward, its epilogue off) gives raw q, k, v of the drafted nodes;
qnre_qkv_norm_rope_append normalises and rotates them and writes K and V into
the paged cache; qnre_tree_attention lets every node attend to its row's tokens
and its ancestors; qnre_verify_tree walks the drafted tree against the model's
probabilities; qnre_cache_compact keeps the accepted path.  The drafter is a table of
next-token distributions.  Prompts enter the same way, as chains of 64 nodes.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ulysses_qkv_proj_gb300 import binding as qb  # noqa: E402


class Model:
    """Random weights; `sharpness` scales the logits."""

    def __init__(self, heads=4, layers=2, vocab=1003, max_positions=4096, sharpness=4.0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.layers, self.vocab = heads, layers, vocab
        self.hidden = hidden = heads * qb.HEAD_DIM

        def randn(*shape, std):
            return (std * torch.randn(shape, generator=gen, device="cuda")).bfloat16()

        self.embed = randn(vocab, hidden, std=1.0)
        self.w_qkv = [randn(hidden, 3 * hidden, std=hidden ** -0.5) for _ in range(layers)]
        self.w_out = [randn(hidden, hidden, std=hidden ** -0.5) for _ in range(layers)]
        self.norms = [(1 + 0.1 * torch.randn((2, qb.HEAD_DIM), generator=gen, device="cuda")).bfloat16()
                      for _ in range(layers)]
        self.head = randn(hidden, vocab, std=sharpness * hidden ** -0.5)
        half = qb.HEAD_DIM // 2
        angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(half, dtype=torch.float64) / half)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        # the drafter knows, for each token, a noisy version of what the model says without context
        self.draft_logits = (self.embed @ self.head).float() + torch.randn((vocab, vocab), generator=gen, device="cuda")


class Decoder:
    """Rows of a paged cache that decode together."""

    def __init__(self, model, rows, max_tokens=1024, page_size=16):
        self.m = model
        blocks = -(-(max_tokens + qb.MAX_NODES) // page_size)
        self.cache = qb.alloc_paged_cache(model.layers, rows * blocks, model.heads, page_size, qb.HEAD_DIM, rows, blocks)
        self.rows = torch.arange(rows, dtype=torch.int32, device="cuda")
        self.plan = qb.Plan(model.hidden, model.heads, 1, max_tokens=rows * qb.MAX_NODES, flags=qb.FLAG_EPILOGUE_OFF)

    def full(self, value):
        return torch.full_like(self.rows, value)

    def forward(self, tokens, parents):
        """Logits [n, nodes, vocab] of drafted nodes (parents None: a chain); their K and V lie behind
        the rows' tokens afterwards."""
        m, cache = self.m, self.cache
        n, nodes = tokens.shape
        qb.qnre_cache_reserve(cache, self.rows, self.full(nodes))
        if parents is None:
            masks, depths = None, torch.arange(nodes, dtype=torch.int32, device="cuda").expand(n, nodes)
        else:
            masks = torch.empty((n, nodes), dtype=torch.int64, device="cuda")
            depths = torch.empty((n, nodes), dtype=torch.int32, device="cuda")
            qb.qnre_tree_masks(parents, masks, depths)
        positions = (cache.seq_lens[:, None] + depths).contiguous()
        x = m.embed[tokens.long()]
        raw = qb.alloc_outputs(self.plan, n, nodes)
        q, out = (torch.empty((n, nodes, m.heads, qb.HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        workspace = qb.tree_attention_workspace(q, cache)
        for layer in range(m.layers):
            qw, kw = m.norms[layer]
            qb.qnre_forward(self.plan, x[None], m.w_qkv[layer], qw, kw, m.cos_sin, None, raw)
            qb.qnre_qkv_norm_rope_append(raw["q"][0], raw["k"][0], raw["v"][0], qw, kw, m.cos_sin, positions, q, cache,
                                         layer, self.rows)
            qb.qnre_tree_attention(q, cache, layer, self.rows, masks, out, workspace=workspace)
            x = x + out.view(n, nodes, -1) @ m.w_out[layer]
        return (x @ m.head).float()

    def prefill(self, prompts):
        """Takes all but the last token of each prompt [n, S] into the cache."""
        for at in range(0, prompts.shape[1] - 1, qb.MAX_NODES):
            part = prompts[:, at:min(at + qb.MAX_NODES, prompts.shape[1] - 1)]
            self.forward(part, None)
            path = torch.arange(part.shape[1], dtype=torch.int32, device="cuda").expand(part.shape).contiguous()
            qb.qnre_cache_compact(self.cache, self.rows, path, self.full(part.shape[1]))

    def draft(self, last, nodes, branch, generator):
        """A tree of `nodes` drafted tokens below each row's last one, children sampled from the table."""
        n = last.numel()
        parents = [-1] + [(i - 1) // branch for i in range(1, nodes)]
        tokens = torch.empty((n, nodes), dtype=torch.int32, device="cuda")
        tokens[:, 0] = last
        for i in range(1, nodes):
            p = torch.softmax(self.m.draft_logits[tokens[:, parents[i]].long()], -1)
            tokens[:, i] = torch.multinomial(p, 1, generator=generator)[:, 0].int()
        draft_probs = torch.softmax(self.m.draft_logits[tokens.long()], -1)
        return tokens, torch.tensor([parents] * n, dtype=torch.int32, device="cuda"), draft_probs

    def step(self, last, nodes, branch, generator, greedy=False):
        """Drafts, verifies and keeps.  Returns the next last tokens and the emitted ones (-1 padded)."""
        tokens, parents, draft_probs = self.draft(last, nodes, branch, generator)
        logits = self.forward(tokens, parents)
        if greedy:
            target = torch.nn.functional.one_hot(logits.argmax(-1), self.m.vocab).float()
        else:
            target = torch.softmax(logits, -1)
        n = last.numel()
        accept = torch.rand((n, nodes), generator=generator, device="cuda")
        sample = torch.rand(n, generator=generator, device="cuda")
        path = torch.empty((n, nodes), dtype=torch.int32, device="cuda")
        counts, following = torch.empty_like(self.rows), torch.empty_like(self.rows)
        qb.qnre_verify_tree(target, draft_probs, tokens, parents, accept, sample, path, counts, following)
        qb.qnre_cache_compact(self.cache, self.rows, path, counts)
        # emitted: the accepted drafts after the root, then the sampled token
        chosen = tokens.gather(1, path.clamp(min=0).long())
        emitted = torch.where(path >= 0, chosen, -1)[:, 1:]
        emitted = torch.cat([emitted, self.full(-1)[:, None]], 1)
        emitted.scatter_(1, counts[:, None].long() - 1, following[:, None])
        return following, emitted


def generate(model, prompts, new_tokens, nodes, branch, greedy=False, seed=0):
    """Tokens [n][...] decoded after the prompts, at least new_tokens each, and the steps it took."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d = Decoder(model, prompts.shape[0], max_tokens=prompts.shape[1] + new_tokens + 2 * nodes)
    d.prefill(prompts)
    last = prompts[:, -1].contiguous()
    texts, steps = [[] for _ in range(prompts.shape[0])], 0
    while min(len(t) for t in texts) < new_tokens:
        last, emitted = d.step(last, nodes, branch, gen, greedy)
        steps += 1
        for t, row in zip(texts, emitted.tolist()):
            t.extend(x for x in row if x >= 0)
        if max(len(t) for t in texts) > new_tokens + nodes:
            break
    if d.cache.status() != 0:
        raise RuntimeError("the cache reported an error")
    return texts, steps


def main():
    model = Model()
    gen = torch.Generator().manual_seed(1)
    prompts = torch.randint(0, model.vocab, (4, 150), generator=gen, dtype=torch.int32).cuda()
    texts, steps = generate(model, prompts, 40, nodes=8, branch=2)
    print(f"sampled: {sum(map(len, texts))} tokens of 4 rows in {steps} steps")
    texts, steps = generate(model, prompts, 40, nodes=8, branch=2, greedy=True)
    print(f"greedy: {sum(map(len, texts))} tokens of 4 rows in {steps} steps")


if __name__ == "__main__":
    main()
