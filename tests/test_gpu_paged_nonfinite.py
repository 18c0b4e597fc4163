"""Infinities and NaN in the paged cache: where the definition in float64 has
them, and nowhere else."""
import pytest
import torch

from tests import _serving_ref as R
from tests.test_gpu_paged import call, make

pytestmark = pytest.mark.gpu


def spoil(x, which, n, pos, value, channel=None):
    """Writes ``value`` to the cache row of position ``pos`` of sequence ``n`` (one channel, or all)."""
    page = x["kp"].shape[1]
    row = x[which][int(x["table"][n, pos // page]), pos % page]
    row[:, slice(None) if channel is None else slice(channel, channel + 1)] = value


def compare(x):
    o, status = call(x)
    assert status == 0
    ref, size = R.attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu"], x["q"].shape[2] ** -0.5)
    R.check(o, ref, R.attention_bar(size), "o")
    got, inf = R.d(o), torch.isinf(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got[inf], ref[inf])
    return o


CHUNKS = [([5], [70], 4, 2), ([140], [140], 1, 1), ([200, 3], [900, 40], 6, 2), ([2], [129], 8, 1), ([9, 4], [6, 257], 4, 2),
          ([20], [40000], 8, 2), ([130], [640], 128, 1), ([64], [64 + 128], 2, 1)]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens,Hq,Hkv", CHUNKS)
def test_values_of_later_tokens_do_not_reach_earlier_rows(new, lens, Hq, Hkv, D, value):
    """A token sees the positions up to its own: what a later one holds as its
    value, whole or in one channel, leaves it alone."""
    x = make(new, lens, Hq, Hkv, D, 16, seed=sum(new) + D)
    clean = compare(x)
    for n, (L, total) in enumerate(zip(new, lens)):
        spoil(x, "vp", n, total - 1, value)
        if min(L, total) > 2:
            spoil(x, "vp", n, total - 2, value, channel=D - 3)
            spoil(x, "vp", n, total - 1 - min(L, total) // 2, -value, channel=5)
    o = compare(x)
    first = x["cu"][0]
    untouched = new[0] - 1 - min(new[0], lens[0]) // 2 if min(new[0], lens[0]) > 2 else new[0] - 1
    assert torch.equal(o[first:first + untouched], clean[first:first + untouched])
    assert not torch.isfinite(o[x["cu"][1] - 1]).any()


@pytest.mark.parametrize("new,lens", [([1], [300]), ([40], [300]), ([2], [40000])])
def test_values_that_every_row_sees(new, lens):
    x = make(new, lens, 4, 2, 128, 16, seed=2)
    spoil(x, "vp", 0, 17, float("inf"), channel=3)
    spoil(x, "vp", 0, 200, float("nan"), channel=90)
    o = compare(x)
    assert torch.isinf(o[..., 3]).all() and torch.isnan(o[..., 90]).all() and torch.isfinite(o[..., :3]).all()


@pytest.mark.parametrize("new,lens", [([1], [1]), ([3], [2]), ([130, 1], [131, 700]), ([1], [40000])])
def test_scores_that_are_all_minus_infinity(new, lens):
    """exp(-inf - (-inf)): NaN, unlike a row that sees no key, which is zero."""
    x = make(new, lens, 4, 2, 64, 16, seed=3)
    x["q"][..., 7] = -1.0
    x["kp"][..., 7] = float("inf")
    o = compare(x)
    assert torch.isnan(o[x["cu"][1] - 1]).all()
    if lens[0] < new[0]:
        assert not o[0].any()
