"""Sizes past 32 bits are refused, not cut (no GPU needed: a size is looked at
before where the tensor is)."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import build as kbuild, decode, norm

BIG = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def huge(*shape, dtype=torch.bfloat16):
    return torch.zeros(1, dtype=dtype).expand(*shape)


def test_norm_width():
    y = huge(1, BIG + 64)
    with pytest.raises(ValueError, match="width"):
        norm.block_norm_fwd(y)
    with pytest.raises(ValueError, match="width"):
        norm.block_norm_bwd(y, dh_out=y)


@pytest.mark.parametrize("shape,name", [((1, BIG + 2, 64), "heads"), ((1, 1, BIG + 64), "head_dim")])
def test_step_and_attention_heads(shape, name):
    t, i = huge(*shape), torch.zeros(2, dtype=torch.int32)
    pages, f = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16), torch.zeros(1)
    with pytest.raises(ValueError, match=name):
        decode.kda_step(t, t, t, t, t, f, f, i, torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError, match=name):
        decode.paged_attention(t, pages, pages, i[:1, None], i[:1], i)
    with pytest.raises(ValueError, match=name):
        decode.paged_append(t, t, pages, pages, i[:1, None], i[:1], i)


def test_step_sequences():
    t, f = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1)
    with pytest.raises(ValueError, match="cu_seqlens"):
        decode.kda_step(t, t, t, t, t, f, f, huge(BIG + 2, dtype=torch.int32), torch.zeros(1, 1, 64, 64))
