"""The block norm's optional buffers: each output may be given by itself, and
a workspace may be given to a call that needs none."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import norm
from tests.test_gpu_norm import make

pytestmark = pytest.mark.gpu


def test_each_output_may_be_given_by_itself():
    x, _, _ = make(20, 64, torch.bfloat16, "zhpn", seed=1)
    kw = {k: x[k] for k in ("z", "h", "w_post", "w_pre")}
    ho, n = norm.block_norm_fwd(x["y"], **kw)
    mine = torch.full_like(n, 7.0)
    a, b = norm.block_norm_fwd(x["y"], **kw, out=(None, mine))
    assert b is mine and torch.equal(mine, n) and torch.equal(a, ho)
    mine = torch.full_like(ho, 7.0)
    a, b = norm.block_norm_fwd(x["y"], **kw, out=(mine, None))
    assert a is mine and torch.equal(mine, ho) and torch.equal(b, n)
    a, b = norm.block_norm_fwd(x["y"], z=x["z"], out=(None, None))
    assert a is not None and b is None
    with pytest.raises((ValueError, RuntimeError)):
        norm.block_norm_fwd(x["y"], z=x["z"], out=(None, mine))  # n without w_pre


def test_a_workspace_where_none_is_needed():
    x, dho, _ = make(20, 64, torch.bfloat16, "zh", seed=2)
    kw = dict(z=x["z"], h=x["h"], dh_out=dho)
    a = norm.block_norm_bwd(x["y"], **kw)
    ws = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    b = norm.block_norm_bwd(x["y"], **kw, workspace=ws)
    assert bool((ws == 7).all()) and all(torch.equal(a[k], b[k]) for k in ("dy", "dz", "dh"))
