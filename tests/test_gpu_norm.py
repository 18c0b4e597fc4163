"""The block norm, forward and backward, against float64 autograd of its
formula and against differences.

Bars: sums are fp32 trees over at most 8192 terms (relative error below 1e-6 of
the sum of magnitudes, itself a few RMS times the term count), so every output
is held to 5e-5 of its RMS beyond its own rounding; a weight gradient adds up
to a few thousand rows the same way."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import norm
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu
BAR = 5e-5


def make(rows, D, dtype, parts, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    x = {"y": rnd(rows, D, std=0.7).to(dtype).cuda()}
    x["z"] = rnd(rows, D, std=2.0).to(dtype).cuda() if "z" in parts else None
    x["h"] = rnd(rows, D, std=2.0).to(dtype).cuda() if "h" in parts else None
    x["w_post"] = (1 + rnd(D, std=0.2)).cuda() if "p" in parts else None
    x["w_pre"] = (1 + rnd(D, std=0.2)).cuda() if "n" in parts else None
    return x, rnd(rows, D).to(dtype).cuda(), rnd(rows, D).to(dtype).cuda() if "n" in parts else None


def reference(x, dho, dn, a, b, eps=1e-5):
    leaf = {k: None if v is None else R.d(v).requires_grad_() for k, v in x.items()}
    ho, n = R.block_norm(*(leaf[k] for k in ("y", "z", "h", "w_post", "w_pre")), a, b, eps)
    loss = 0 if dho is None else (ho * R.d(dho)).sum()
    if dn is not None:
        loss = loss + (n * R.d(dn)).sum()
    names = [k for k, v in leaf.items() if v is not None]
    grads = torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True)
    return ho.detach(), None if n is None else n.detach(), dict(zip(names, grads))


def compare(x, dho, dn, a, b):
    kw = dict(residual_scale=a, block_scale=b, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})
    ho, n = norm.block_norm_fwd(x["y"], **kw)
    g = norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, **kw)
    r_ho, r_n, r_g = reference(x, dho, dn, a, b)
    R.check(ho, r_ho, BAR, "h_out")
    assert (n is None) == (r_n is None)
    if n is not None:
        R.check(n, r_n, BAR, "n")
    for k in ("y", "z", "h", "w_post", "w_pre"):
        assert (g["d" + k] is None) == (x[k] is None)
        if x[k] is not None:
            R.check(g["d" + k], torch.zeros_like(R.d(x[k])) if r_g[k] is None else r_g[k], BAR, "d" + k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64), (1000, 128), (17, 129), (9, 200), (64, 512), (33, 1000),
                                    (4, 1537), (700, 2048), (3, 4096), (5, 4097), (2, 8191), (6, 8192)])
def test_every_part(rows, D, dtype):
    x, dho, dn = make(rows, D, dtype, "zhpn", seed=rows + D)
    compare(x, dho, dn, 0.9, 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(9001, 3), (30000, 65), (5003, 130), (3000, 257), (1501, 1001), (1300, 2050),
                                    (700, 4093), (400, 8189), (321, 8186)])
def test_odd_widths_with_several_rows_a_group(rows, D, dtype):
    """More rows than groups are resident: a group's rows keep their shift."""
    x, dho, dn = make(rows, D, dtype, "zhpn", seed=rows)
    compare(x, dho, dn, 0.9, 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts", ["", "p", "z", "zp", "h", "hp", "hn", "n", "zn", "zhn", "hpn"])
@pytest.mark.parametrize("rows,D", [(300, 128), (40, 1024), (7, 33)])
def test_parts_left_out(rows, D, parts, dtype):
    x, dho, dn = make(rows, D, dtype, parts, seed=rows)
    compare(x, dho, dn, 1.25, -0.75)


@pytest.mark.parametrize("which", ["dh_out", "dn"])
def test_one_gradient_only(which):
    x, dho, dn = make(50, 256, torch.float32, "zhpn", seed=2)
    compare(x, dho if which == "dh_out" else None, dn if which == "dn" else None, 1.0, 1.0)


def test_gradient_against_differences():
    """Central differences of the kernel's own fp32 forward in random
    directions of length 1: the step of 1e-2 leaves a third-order remainder below
    1e-4, and fp32 outputs give about 1e-6 / 1e-2: within 1e-2 of the gradient's size."""
    x, dho, dn = make(6, 40, torch.float32, "zhpn", seed=7)
    kw = dict(residual_scale=0.9, block_scale=0.5)
    g = norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, **kw, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})

    def loss(v):
        ho, n = norm.block_norm_fwd(v["y"], **kw, **{k: v[k] for k in ("z", "h", "w_post", "w_pre")})
        return (ho.double() * dho.double()).sum() + (n.double() * dn.double()).sum()

    gen = torch.Generator().manual_seed(3)
    for k in ("y", "z", "h", "w_post", "w_pre"):
        dirn = torch.randn(x[k].shape, generator=gen).cuda()
        dirn = dirn / dirn.norm()
        up, down = dict(x), dict(x)
        up[k], down[k] = x[k] + 1e-2 * dirn, x[k] - 1e-2 * dirn
        num = (loss(up) - loss(down)).item() / 2e-2
        ana = (g["d" + k].double() * dirn.double()).sum().item()
        assert abs(num - ana) <= 1e-2 * max(1.0, g["d" + k].norm().item()), (k, num, ana)


def test_autograd_wrapper_and_leading_dimensions():
    x, dho, dn = make(24, 64, torch.bfloat16, "zhpn", seed=4)
    v = {k: (t.view(4, 6, 64) if t.dim() == 2 else t).detach().requires_grad_() for k, t in x.items()}
    ho, n = norm.block_norm(v["y"], z=v["z"], h=v["h"], w_post=v["w_post"], w_pre=v["w_pre"], residual_scale=0.9,
                            block_scale=0.5)
    (n.float() * dn.view(4, 6, 64).float()).sum().backward()  # h_out unused: its gradient is None
    _, _, r = reference(x, None, dn, 0.9, 0.5)
    for k, t in v.items():
        R.check(t.grad.view(x[k].shape), r[k], BAR, k)
    u = norm.block_norm(x["y"], z=x["z"], w_post=x["w_post"])
    R.check(u, reference({**x, "h": None, "w_pre": None}, dho, None, 1.0, 1.0)[0], BAR, "u")


@pytest.mark.parametrize("D", [512, 517])
def test_in_place_buffers_and_no_rows(D):
    x, dho, dn = make(3000, D, torch.bfloat16, "zhpn", seed=5)
    kw = dict(residual_scale=0.9, block_scale=0.5, **{k: x[k] for k in ("z", "w_post", "w_pre")})
    ho, n = norm.block_norm_fwd(x["y"], h=x["h"], **kw)
    h = x["h"].clone()
    ho2, n2 = norm.block_norm_fwd(x["y"], h=h, out=(h, torch.empty_like(h)), **kw)
    assert torch.equal(ho, ho2) and torch.equal(n, n2) and ho2 is h
    e = torch.empty(0, D, dtype=torch.bfloat16).cuda()
    ho, n = norm.block_norm_fwd(e, w_pre=x["w_pre"])
    assert ho.shape == n.shape == (0, D)
    g = norm.block_norm_bwd(e, w_pre=x["w_pre"], dn=e)
    assert not g["dw_pre"].any()


def test_neighbouring_rows_do_not_touch_each_other():
    """Rows of an odd width share 16-byte vectors: NaN and infinities stay in their row."""
    x, dho, dn = make(2000, 129, torch.bfloat16, "zhpn", seed=11)
    kw = dict(residual_scale=0.9, block_scale=0.5)
    clean = norm.block_norm_fwd(x["y"], **kw, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})
    grads = norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, **kw, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})
    bad = torch.arange(1, 2000, 3).cuda()
    for t in (x["y"], x["z"], x["h"], dho, dn):
        t[bad] = float("nan")
    out = norm.block_norm_fwd(x["y"], **kw, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})
    g = norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, **kw, **{k: x[k] for k in ("z", "h", "w_post", "w_pre")})
    good = torch.ones(2000, dtype=torch.bool).cuda()
    good[bad] = False
    for a, b in [*zip(clean, out), *((grads[k], g[k]) for k in ("dy", "dz", "dh"))]:
        assert torch.equal(a[good], b[good]) and torch.isnan(b[bad]).all()


def test_extreme_rows():
    """Zero rows, rows of the dtype's large values, saturated gates, an infinity."""
    x, dho, dn = make(6, 128, torch.float32, "zhpn", seed=6)
    x["y"][0] = 0
    x["y"][1] *= 1e15
    x["y"][2] *= 1e-15
    x["z"][3, ::2], x["z"][3, 1::2] = 200.0, -200.0
    compare(x, dho, dn, 0.9, 0.5)
    x["y"][4, 5] = float("inf")
    x["z"][5, 7] = float("nan")
    ho, n = norm.block_norm_fwd(x["y"], z=x["z"], h=x["h"], w_post=x["w_post"], w_pre=x["w_pre"])
    r_ho, r_n, _ = reference(x, dho, dn, 1.0, 1.0)
    assert torch.equal(torch.isnan(ho).cpu(), torch.isnan(r_ho)) and torch.equal(torch.isnan(n).cpu(), torch.isnan(r_n))


def test_same_bits_every_run():
    x, dho, dn = make(5000, 128, torch.bfloat16, "zp", seed=8)
    kw = dict(z=x["z"], w_post=x["w_post"], dh_out=dho)
    a, b = norm.block_norm_bwd(x["y"], **kw), norm.block_norm_bwd(x["y"], **kw)
    assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)
