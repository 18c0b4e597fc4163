"""Packed attention of many short sequences: more items of one kind than there are SMs, so that each CTA takes
several in a row, among them sequences with an odd number of 128-row tiles, whose last item has one stream."""
import pytest
import torch

import _blocks_ref as R
from test_gpu_packed_attention import inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hk", [
    ([257 + 53 * i % 128 for i in range(40)], 16, 4),          # one stream of three key tiles, 640 of them
    ([300], 200, 25),                                          # the same of one sequence
    ([513 + 37 * i % 128 for i in range(12)], 32, 8),          # one stream of five
    ([100 + 71 * i % 300 for i in range(50)], 16, 4),          # one of one or three, or two
    ([700, 320, 64, 300, 900, 310, 1, 128, 129, 383] * 2, 24, 8),
])
def test_many_short_sequences(lens, Hq, Hk, D):
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=len(lens))
    got = run(q, k, v, d_o, cu)
    R.check_all(got, *R.attention(q, k, v, cu.tolist(), D ** -0.5, d_o))
    for _ in range(10):  # CTAs come to their items in other orders
        again = run(q, k, v, d_o, cu)
        assert all(torch.equal(again[n], got[n]) for n in got)


@pytest.mark.parametrize("D", [64, 128])
def test_short_sequences_with_rising_maxima(D):
    """Outputs rescaled at every tile of items of one stream that follow one another."""
    lens, Hq, Hk = [384, 300, 640, 257] * 8, 8, 4
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=D, std=0.5)
    u = torch.ones(D, device="cuda") * D ** -0.5
    at = torch.cat([torch.arange(n) for n in lens]).cuda().float()
    q = (q.float() + 3.0 * u).to(torch.bfloat16)
    k = (k.float() + 0.25 * at[:, None, None] * u).to(torch.bfloat16)
    R.check_all(run(q, k, v, d_o, cu, 0.125), *R.attention(q, k, v, cu.tolist(), 0.125, d_o))
