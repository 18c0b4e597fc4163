"""Verification of drafted tokens against the plain implementation: tokens and
counts are equal. The exact-tie cases use dyadic values, where every product,
difference and quotient is exact; elsewhere seeds are fixed."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import decode, kda as K
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu


def make(N, T, V, seed=0, draft=True):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(N, T + 1, V, generator=g) * 2
    x = {"target": torch.softmax(logits, -1)}
    x["draft"] = torch.softmax(logits[:, :T] + 0.5 * torch.randn(N, T, V, generator=g), -1) if draft else None
    x["x"] = torch.distributions.Categorical(probs=(x["draft"] if draft else x["target"][:, :T]).reshape(-1, V)).sample() \
        .view(N, T).to(torch.int32) if T else torch.zeros(N, 0, dtype=torch.int32)
    x["num"] = torch.randint(0, T + 1, (N,), generator=g, dtype=torch.int32)
    x["u"] = torch.rand(N, T, generator=g)
    x["noise"] = torch.empty(N, V).exponential_(generator=g).clamp_min(1e-20)
    return x


def compare(x, **kw):
    dev = {k: None if v is None else v.cuda() for k, v in x.items()}
    tokens, accepted = decode.verify_drafts(dev["target"], dev["draft"], dev["x"], dev["num"], dev["u"], dev["noise"], **kw)
    rt, ra = R.verify(x["target"], x["draft"], x["x"], x["num"], x["u"], x["noise"])
    assert torch.equal(accepted.cpu().long(), ra), (accepted.tolist(), ra.tolist())
    assert torch.equal(tokens.cpu().long(), rt)
    return tokens, accepted


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("N,T,V", [(1, 1, 1), (1, 3, 1000), (7, 5, 1001), (20, 8, 4096), (3, 40, 130), (2, 2, 50001),
                                   (5, 0, 333), (2, 1, 100000)])
def test_against_plain(N, T, V, draft):
    torch.manual_seed(N + V)
    compare(make(N, T, V, seed=N * 100 + T, draft=draft))


def test_all_accepted_all_refused_and_no_counts():
    x = make(6, 4, 500, seed=3)
    x["num"] = None
    x["u"].zero_()
    _, accepted = compare(x)
    assert accepted.tolist() == [4] * 6
    x["u"].fill_(0.999)
    x["target"].scatter_(2, torch.cat([x["x"], x["x"][:, :1]], 1).long()[..., None], 0.0)
    _, accepted = compare(x)
    assert accepted.tolist() == [0] * 6


@pytest.mark.parametrize("V", [64, 77])
def test_ties_take_the_lowest_index(V):
    x = {"target": torch.full((2, 2, V), 1 / 64), "draft": torch.full((2, 1, V), 1 / 128), "x": torch.zeros(2, 1, dtype=torch.int32),
         "num": torch.tensor([1, 0], dtype=torch.int32), "u": torch.full((2, 1), 0.5), "noise": torch.full((2, V), 0.5)}
    x["target"][0, 0, 0] = 1 / 512  # 0.5 / 128 is above it: refused, and nothing left at 0
    tokens, accepted = compare(x)
    assert tokens[:, 0].tolist() == [1, 0] and accepted.tolist() == [0, 0]
    x["u"].fill_(0.25)  # equal products are refused: u q < p is strict
    x["target"][0, 0, 0] = 1 / 512
    assert compare(x)[1].tolist() == [0, 0]


def test_nothing_left_falls_back_to_the_target():
    x = make(3, 2, 100, seed=5)
    x["num"] = torch.tensor([2, 2, 2], dtype=torch.int32)
    x["target"][:, 0] = x["draft"][:, 0]  # p = q: accepted unless u q >= p
    x["u"][:, 0] = 1.0
    tokens, accepted = compare(x)
    assert accepted.tolist() == [0, 0, 0] and bool((tokens[:, 0] >= 0).all())
    x["target"].zero_()
    tokens, accepted = compare(x)
    assert tokens[:, 0].tolist() == [0, 0, 0]


def test_infinities_and_nan():
    x = make(4, 2, 90, seed=6)
    x["num"] = torch.full((4,), 2, dtype=torch.int32)
    nan = float("nan")
    x["target"][0, 0, int(x["x"][0, 0])] = nan      # refused
    x["draft"][1, 0, int(x["x"][1, 0])] = float("inf")
    x["target"][2, 0, 5] = nan                       # does not count as a candidate
    x["u"][2, 0] = 1.0
    x["target"][3, :, 7] = float("inf")
    x["u"][3] = 0.0
    compare(x)


def test_bad_tokens_and_counts():
    x = make(3, 3, 64, seed=7)
    x["num"] = torch.tensor([3, 9, -4], dtype=torch.int32)
    x["x"][0, 0], x["x"][1, 1] = 64, -1
    x["u"].zero_()
    for draft in (x["draft"], None):
        x["draft"] = draft
        status = torch.zeros(1, dtype=torch.int32).cuda()
        _, accepted = compare(x, status=status)
        assert accepted.tolist() == [0, 1, 0] and K.query_device_status(status) == 6


def test_offsets_past_32_bits():
    N, T, V = 3, 7, 1 << 27  # the target has 3 * 2^30 elements
    target = torch.zeros(N, T + 1, V, device="cuda")
    noise = torch.ones(N, V, device="cuda")
    x = torch.arange(T, dtype=torch.int32).repeat(N, 1).cuda()
    target[:, torch.arange(T), torch.arange(T)] = 1.0
    target[:, T, V - 2:] = 1.0
    tokens, accepted = decode.verify_drafts(target, None, x, None, torch.zeros(N, T, device="cuda"), noise)
    assert accepted.tolist() == [T] * N and tokens[:, T].tolist() == [V - 2] * N and torch.equal(tokens[:, :T], x)


def test_distribution_of_the_next_token():
    """One draft, many sequences: the next token is distributed as the target
    (5 standard deviations of a multinomial count)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    N, V = 20000, 5
    p, q = torch.tensor([0.4, 0.1, 0.2, 0.25, 0.05]), torch.tensor([0.1, 0.5, 0.2, 0.1, 0.1])
    x = torch.multinomial(q.cuda(), N, True, generator=g).to(torch.int32)[:, None]
    tokens, accepted = decode.verify_drafts(
        p.cuda().expand(N, 2, V).contiguous(), q.cuda().expand(N, 1, V).contiguous(), x, None,
        torch.rand(N, 1, device="cuda", generator=g), torch.empty(N, V, device="cuda").exponential_(generator=g))
    count = torch.bincount(tokens[:, 0].long(), minlength=V).cpu().double()
    assert bool(((count - N * p).abs() <= 5 * (N * p * (1 - p)).sqrt()).all()), count
    rate = accepted.double().mean().item()
    a = torch.minimum(p, q).sum().item()
    assert abs(rate - a) <= 5 * (a * (1 - a) / N) ** 0.5
