"""Calls one behind another whose kernels overlap: each sees what the one before has written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_verification_reads_the_probabilities_just_filtered():
    """Both distributions made and verified in one captured graph, with new logits at each replay; what separate calls give."""
    from ulysses_qkv_proj_gb300 import binding as qb
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, N, V = 5, 4, 32003
    logits, drafts = (torch.empty((n, N, V), device="cuda") for _ in range(2))
    target, draft = (torch.zeros((n, N, V), device="cuda") for _ in range(2))
    k = _i32([3, 50, 1, 0, 9])
    tokens, parents = torch.zeros((n, N), dtype=torch.int32, device="cuda"), _i32([[-1, 0, 1, 2]] * n)
    accept, pick = torch.rand((n, N), generator=gen, device="cuda"), torch.rand(n, generator=gen, device="cuda")

    def outputs():
        return torch.full((n, N), -7, dtype=torch.int32, device="cuda"), *(torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(2))

    def calls(out, between=lambda: None):
        qb.qnre_filter_probs(logits, target, top_k=k)
        between()
        qb.qnre_filter_probs(drafts, draft, top_k=k)
        between()
        qb.qnre_verify_tree(target, draft, tokens, parents, accept, pick, *out)

    def refill():
        logits.normal_(generator=gen)
        drafts.copy_(logits + 0.3 * torch.randn(logits.shape, generator=gen, device="cuda"))
        tokens[:, 1:] = drafts[:, :-1].argmax(-1).int()

    refill()
    out, graph, s = outputs(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    calls(out)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            calls(out)
    accepted = 0
    for _ in range(12):
        refill()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = outputs()
        calls(want, torch.cuda.synchronize)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        accepted += int((got[1] > 1).sum())
    assert accepted > 0
