"""The block norm far from 1: rows whose squares are near the ends of fp32,
and gates at minus infinity, against float64 autograd of the formula."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import norm
from tests import _serving_ref as R
from tests.test_gpu_norm import BAR, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e13, 1e-5), (1e15, 1e-5), (1e17, 1e-5), (1e-13, 0.0), (1e-15, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("rows,D", [(40, 256), (9, 129), (3, 4096)])
def test_gradients_of_large_and_small_rows(rows, D, size, eps, dtype):
    """The residual stream and the block's output scaled by ``size`` (whose square is
    in fp32's range): the gradients are those of the plain size over ``size``."""
    x, _, dn = make(rows, D, dtype, "zhpn", seed=D)
    x["h"] = x["h"] * size
    kw = dict(residual_scale=0.9, block_scale=0.5 * size, eps=eps)
    tensors = {k: x[k] for k in ("z", "h", "w_post", "w_pre")}
    ho, n = norm.block_norm_fwd(x["y"], **kw, **tensors)
    g = norm.block_norm_bwd(x["y"], dn=dn, **kw, **tensors)
    r_ho, r_n, r_g = reference(x, None, dn, 0.9, 0.5 * size, eps)
    R.check(ho, r_ho, BAR, "h_out")
    R.check(n, r_n, BAR, "n")
    for k in ("y", "z", "h", "w_post", "w_pre"):
        R.check(g["d" + k], r_g[k], BAR, "d" + k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts,D", [("zp", 128), ("zhpn", 128), ("zhpn", 4096), ("zhpn", 77)])
def test_a_gate_of_minus_infinity_is_closed(parts, D, dtype):
    """sigmoid(-inf) is 0, and so is its derivative."""
    x, dho, dn = make(12, D, dtype, parts, seed=D)
    shut = R.inf_like(x["z"]).neg()
    kw = dict(residual_scale=0.9, block_scale=0.5, **{k: x[k] for k in ("h", "w_post", "w_pre")})
    ho, _ = norm.block_norm_fwd(x["y"], z=shut, **kw)
    g = norm.block_norm_bwd(x["y"], z=shut, dh_out=dho, dn=dn, **kw)
    assert torch.equal(ho, torch.zeros_like(ho) if x["h"] is None else (x["h"].float() * 0.9).to(dtype))
    assert not g["dy"].any() and not g["dz"].any() and not g["dw_post"].any()
    mixed = x["z"].clone()
    mixed[:, ::3] = -float("inf")
    mixed[:, 1::3] = -88.0
    x["z"] = mixed
    g = norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, z=mixed, **kw)
    r_ho, _, r_g = reference(dict(x, z=mixed.clamp_min(-1e4)), dho, dn, 0.9, 0.5)
    R.check(norm.block_norm_fwd(x["y"], z=mixed, **kw)[0], r_ho, BAR, "h_out")
    for k in ("y", "z", "w_post"):
        R.check(g["d" + k], r_g[k], BAR, "d" + k)
