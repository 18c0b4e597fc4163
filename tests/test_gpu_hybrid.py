"""The example stack: training lowers the loss, and decoding with drafted
tokens gives the tokens of decoding without them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss():
    from recompute_kda_chunkwise_gb300 import hybrid
    torch.manual_seed(1)
    model = hybrid.Stack(seed=3)
    tokens = torch.randint(0, 512, (300,), device="cuda")
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    losses = [hybrid.train_step(model, tokens, cu, tokens.roll(-1), lr=1e-2).item() for _ in range(4)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("kinds", [("delta", "delta"), ("delta", "attn", "delta")])
def test_drafts_do_not_change_greedy_decoding(kinds):
    """Where the two differ, the likeliest tokens must have been as good as
    tied (bf16 activations of calls of different lengths may round apart)."""
    from recompute_kda_chunkwise_gb300 import hybrid
    model = hybrid.Stack(kinds=kinds, seed=5, heads=2, kv_heads=1)
    prompts = [[5, 6, 7, 8] * 10, [1, 2, 3] * 30, [9]]
    plain, calls = hybrid.generate(hybrid.Server(model, 3, 200), prompts, steps=20, drafts=0, greedy=True)
    drafted, fewer = hybrid.generate(hybrid.Server(model, 3, 200), prompts, steps=20, drafts=4, greedy=True)
    assert calls == 19 and fewer <= calls
    for p, a, b in zip(prompts, plain, drafted):
        n = min(len(a), len(b))
        i = next((i for i in range(n) if a[i] != b[i]), None)
        if i is not None:
            probs = hybrid.Server(model, 1, 200).run(torch.tensor(a[:i], device="cuda"), [i])[-1]
            assert abs(probs[a[i]].item() / probs[b[i]].item() - 1) < 0.05, (i, a[i], b[i])


def test_prefill_in_two_parts_equals_one():
    from recompute_kda_chunkwise_gb300 import hybrid
    model = hybrid.Stack(kinds=("delta", "attn"), seed=7, heads=2, kv_heads=2)
    tokens = torch.arange(90, device="cuda") * 7 % 512
    whole = hybrid.Server(model, 1, 96).run(tokens, [90])
    server = hybrid.Server(model, 1, 96)
    server.run(tokens[:40], [40])
    rest = server.run(tokens[40:], [50])
    assert (whole[40:] - rest).abs().max().item() <= 0.05 * whole[40:].max().item()
