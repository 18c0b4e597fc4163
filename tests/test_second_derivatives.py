"""Differentiating a wrapper's gradient is refused: the backward kernels are
not differentiable, and their part of a second derivative must not be dropped
without a word. The kernels are stood in for by elementwise functions here (no
GPU needed)."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import kda as K, norm


def second_derivative(out, leaf):
    """d/d leaf of |d out / d leaf|^2 + |leaf|^2: a loss with a path past the wrapper."""
    (grad,) = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
    (grad.square().sum() + leaf.square().sum()).backward()


def test_block_norm(monkeypatch):
    monkeypatch.setattr(norm, "block_norm_fwd", lambda y, **kw: (y * 2, None))
    monkeypatch.setattr(norm, "block_norm_bwd", lambda y, dh_out=None, **kw: dict(
        dy=dh_out * 2, dz=None, dh=None, dw_post=None, dw_pre=None))
    y = torch.ones(3, 4, requires_grad=True)
    (g,) = torch.autograd.grad(norm.block_norm(y).sum(), y)
    assert bool((g == 2).all())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        second_derivative(norm.block_norm(y), y)


def test_block_norm_with_the_next_norm(monkeypatch):
    monkeypatch.setattr(norm, "block_norm_fwd", lambda y, **kw: (y * 2, y * 3))
    monkeypatch.setattr(norm, "block_norm_bwd", lambda y, dh_out=None, dn=None, **kw: dict(
        dy=(0 if dh_out is None else dh_out * 2) + (0 if dn is None else dn * 3), dz=None, dh=None, dw_post=None, dw_pre=None))
    y = torch.ones(3, 4, requires_grad=True)
    for which, want in ((0, 2.0), (1, 3.0)):  # the other gradient is None
        (g,) = torch.autograd.grad(norm.block_norm(y, w_pre=torch.ones(4))[which].sum(), y)
        assert bool((g == want).all())
        with pytest.raises(RuntimeError, match="once_differentiable"):
            second_derivative(norm.block_norm(y, w_pre=torch.ones(4))[which], y)


@pytest.mark.parametrize("final_state", [False, True])
@pytest.mark.parametrize("gdn2", [False, True])
def test_delta_rule(monkeypatch, gdn2, final_state):
    state = torch.zeros(1)

    def fwd(q, *rest, final_state=False, **kw):
        return (q * 2, state, state + 0) if final_state else (q * 2, state)

    def bwd(q, *rest, **kw):  # ..., cu_seqlens, dO, ctx
        return {**dict.fromkeys(("dk", "dv", "dg", "dbeta", "derase", "dwrite", "dA_log", "ddt_bias")), "dq": rest[-2] * 2}

    monkeypatch.setattr(K, "gdn2_fwd" if gdn2 else "kda_fwd", fwd)
    monkeypatch.setattr(K, "gdn2_bwd" if gdn2 else "kda_bwd", bwd)
    q = torch.ones(2, 3, 4, requires_grad=True)
    one, cu = torch.zeros(1), torch.tensor([0, 2], dtype=torch.int32)

    def call():
        r = K.gdn2(q, one, one, one, one, one, one, one, cu, output_final_state=final_state) if gdn2 else \
            K.kda(q, one, one, one, one, one, one, cu, output_final_state=final_state)
        return r[0] if final_state else r

    (g,) = torch.autograd.grad(call().sum(), q)
    assert bool((g == 2).all())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        second_derivative(call(), q)
