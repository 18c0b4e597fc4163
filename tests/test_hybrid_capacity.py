"""The example's server refuses what its cache does not hold (no GPU needed:
lengths are looked at before any kernel)."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import hybrid


def server(kinds, sequences=2, max_len=40):
    return hybrid.Server(hybrid.Stack(kinds=kinds, dim=64, head_dim=64, vocab=16, device="cpu"), sequences, max_len, page=16)


def test_a_sequence_longer_than_its_pages_is_refused():
    s = server(("delta", "attn"))
    assert s.capacity == 48  # whole pages
    with pytest.raises(ValueError, match="sequence 1 .*49.*48"):
        s.run(torch.zeros(50, dtype=torch.int64), [1, 49])
    s.committed = [0, 47]
    with pytest.raises(ValueError, match="sequence 1 .*49.*48"):
        s.run(torch.zeros(3, dtype=torch.int64), [1, 2], [0, 0])
    assert s.committed == [0, 47]


def test_states_have_no_length():
    assert server(("delta", "delta")).capacity is None


class Fake:
    """A server whose model always continues a token by the next one of 8; records what it is fed."""

    def __init__(self, n, capacity):
        self.m = torch.nn.Module()
        self.m.embed = torch.zeros(8, 1)
        self.table = torch.zeros(n, 1)
        self.capacity, self.committed, self.calls = capacity, [0] * n, []

    def run(self, tokens, lengths, commit=None):
        assert all(c + l <= (self.capacity or 1 << 30) for c, l in zip(self.committed, lengths)), (self.committed, lengths)
        self.calls.append(lengths)
        self.committed = [c + k for c, k in zip(self.committed, lengths if commit is None else commit)]
        return torch.nn.functional.one_hot((tokens + 1) % 8, 8).float()


def verify(target, draft, x, num, u, noise):
    """Greedy verification in plain Python."""
    N, T1, _ = target.shape
    tokens, accepted = torch.full((N, T1), -1), torch.zeros(N, dtype=torch.int64)
    for n in range(N):
        a, most = 0, T1 - 1 if num is None else int(num[n])
        while a < most and target[n, a, x[n, a]] > 0:
            tokens[n, a] = x[n, a]
            a += 1
        tokens[n, a] = target[n, a].argmax()
        accepted[n] = a
    return tokens, accepted


@pytest.mark.parametrize("drafts", [0, 3])
@pytest.mark.parametrize("capacity", [None, 40, 36, 33, 31])
def test_a_sequence_that_runs_ahead_stops_at_its_pages(monkeypatch, capacity, drafts):
    """One prompt repeats and its drafts are accepted; another has none. The first is done long before the second, and
    must not run out of its pages meanwhile."""
    monkeypatch.setattr(hybrid.decode, "verify_drafts", verify)
    prompts = [[0, 1, 2, 3, 4, 5, 6, 7] * 2, [3]]
    s = Fake(2, capacity)
    out, calls = hybrid.generate(s, prompts, steps=16, drafts=drafts, greedy=True)
    for o, p in zip(out, prompts):
        assert o[:len(p)] == p and len(o) - len(p) >= 16
        assert all(b == (a + 1) % 8 for a, b in zip(o[len(p) - 1:], o[len(p):]))
    assert calls == len(s.calls) - 1


def test_too_few_pages_for_the_steps_are_refused(monkeypatch):
    monkeypatch.setattr(hybrid.decode, "verify_drafts", verify)
    with pytest.raises(ValueError, match="16 more tokens"):
        hybrid.generate(Fake(2, 30), [[0, 1, 2, 3, 4, 5, 6, 7] * 2, [3]], steps=16, drafts=3, greedy=True)
