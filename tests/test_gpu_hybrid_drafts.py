"""Drafts that are accepted, several a call: the states and the cache of the
example's server keep exactly the verified tokens."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", [("delta", "delta"), ("delta", "attn", "delta")])
def test_accepted_drafts_save_calls(kinds, monkeypatch):
    """Blocks that add little to the embedding: the likeliest token is the last
    one again, by far, so four drafts of it are right and a call yields five tokens."""
    from recompute_kda_chunkwise_gb300 import hybrid
    monkeypatch.setattr(hybrid, "lookup_drafts", lambda tokens, most: tokens[-1:] * most)
    model = hybrid.Stack(kinds=kinds, seed=5, heads=2, kv_heads=1)
    with torch.no_grad():
        for b in model.blocks:
            b.post.mul_(1e-2)
    prompts = [[5, 6, 7, 7], [1, 1, 1], [9, 9]]
    plain, calls = hybrid.generate(hybrid.Server(model, 3, 64), prompts, steps=20, drafts=0, greedy=True)
    drafted, fewer = hybrid.generate(hybrid.Server(model, 3, 64), prompts, steps=20, drafts=4, greedy=True)
    assert calls == 19 and fewer == 4
    for p, a, b in zip(prompts, plain, drafted):
        n = min(len(a), len(b))
        assert a[:n] == b[:n] and set(a[len(p):]) == {p[-1]}


def test_a_sequence_that_runs_ahead_does_not_outgrow_its_pages():
    from recompute_kda_chunkwise_gb300 import hybrid
    model = hybrid.Stack(kinds=("delta", "attn"), seed=5, heads=2, kv_heads=1)
    prompts = [[5, 6, 7, 8] * 10, [1, 2, 3] * 10, [9]]
    server = hybrid.Server(model, 3, 64)
    out, _ = hybrid.generate(server, prompts, steps=20, drafts=4, greedy=True)
    assert all(len(o) - len(p) >= 20 for o, p in zip(out, prompts)) and max(server.committed) <= server.capacity
