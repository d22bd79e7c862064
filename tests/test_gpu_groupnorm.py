"""The group norm on the GPU against its 64-bit form (tests/gated_ref.py)."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def up(t):
    return t.to(device()) if t is not None else None


def rand(g, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def inputs(rows, groups, size, act, dtype, affine=True, seed=0, mean=0.3):
    g = torch.Generator().manual_seed(31 * seed + rows + 7 * size + groups)
    dim = groups * size
    return dict(x=rand(g, rows, dim, dtype=dtype, mean=mean), weight=rand(g, dim, mean=1.0, std=0.3) if affine else None,
                bias=rand(g, dim, std=0.3) if affine else None, z=rand(g, rows, dim, dtype=dtype) if "gate" in act else None), \
        rand(g, rows, dim, dtype=dtype)


def check(c, dy, groups, act, center, eps):
    ref = R.groupnorm(c["x"], c["weight"], c["bias"], groups, c["z"], act, center, eps, dy)
    a = dict(groups=groups, z=up(c["z"]), act=act, center=center, eps=eps)
    got = dict(y=m3.mamba3_groupnorm_fwd(up(c["x"]), up(c["weight"]), up(c["bias"]), **a),
               **m3.mamba3_groupnorm_bwd(up(c["x"]), up(c["weight"]), up(c["bias"]), dy=up(dy), **a))
    assert set(got) == {"y", "dx"} | {k for k, n in (("dz", "z"), ("dweight", "weight"), ("dbias", "bias")) if c[n] is not None}
    for k in got:
        assert got[k].shape == ref[k][0].shape and not got[k].isnan().any(), k
    worst = {k: R.off(got[k], ref[k]) for k in got}
    note("  " + " ".join(f"{k} {v:.2f}" for k, v in worst.items()))
    assert max(worst.values()) <= 1, worst
    return got


SHAPES = [  # rows, groups, size
    (5, 3, 1), (7, 4, 2), (3, 70, 3), (9, 5, 7), (1, 1, 8), (6, 130, 8), (4, 3, 12), (11, 16, 16), (5, 7, 20),
    (3, 9, 33), (130, 16, 64), (33, 5, 96), (2, 3, 100), (70, 16, 128), (9, 3, 129), (17, 2, 256), (3, 3, 257),
    (5, 1, 511), (40, 2, 512), (3, 2, 513), (5, 1, 520), (4, 3, 1000), (6, 1, 2048), (2, 2, 2049), (3, 1, 2056),
    (3, 1, 4096), (2, 1, 8191), (3, 1, 8192),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act", ["none", "silu", "gate", "pregate"])
def test_groupnorm(shape, act, dtype):
    rows, groups, size = shape
    note(f"group norm {shape} {act} {dtype}")
    center = (rows + groups + size) % 2 == 0
    for cen in (center, not center):
        # a centered group of one value is its bias: it has no deviation
        check(*inputs(rows, groups, size, act, dtype, affine=cen == center), groups, act, cen, 1e-5)


@pytest.mark.parametrize("act", ["none", "gate"])
def test_many_rows(act):
    """More rows than workgroups, so that a workgroup walks several."""
    for shape in ((5000, 2, 64), (2500, 1, 640), (1500, 1, 3000), (4500, 3, 5)):
        note(f"group norm {shape} {act}")
        check(*inputs(*shape, act, BF16), shape[1], act, True, 1e-5)


def test_far_mean():
    """Groups a thousand deviations from zero."""
    for size in (64, 1000):
        check(*inputs(20, 2, size, "none", F32, mean=1000.0), 2, "none", True, 1e-5)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e17, 1e30])
@pytest.mark.parametrize("size", [24, 600])
def test_out_of_range_squares(scale, size, center):
    """Values whose squares leave fp32's range, next to groups in range."""
    c, dy = inputs(9, 4, size, "none", F32)
    c["x"].view(9, 4, size)[::2, 1:3] *= scale
    check(c, dy, 4, "none", center, 0.0)


def test_rows_without_values():
    """A group of zeros has no direction: its norm is its bias. A NaN stays in its group."""
    c, dy = inputs(6, 4, 32, "none", BF16)
    c["x"].view(6, 4, 32)[2, 1] = 0
    got = check(c, dy, 4, "none", True, 1e-5)
    assert torch.equal(got["y"].view(6, 4, 32)[2, 1].cpu(), c["bias"].view(4, 32)[1].bfloat16())
    c["x"].view(6, 4, 32)[3, 2, 5] = float("nan")
    c["x"].view(6, 4, 32)[4, 0, 5] = float("inf")
    y = m3.mamba3_groupnorm_fwd(up(c["x"]), up(c["weight"]), up(c["bias"]), groups=4).view(6, 4, 32)
    bad = y.isnan().any(-1)
    want = torch.zeros(6, 4, dtype=torch.bool)
    want[3, 2] = want[4, 0] = True
    assert torch.equal(bad.cpu(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [32, 13, 700])
def test_views_and_guards(dtype, size):
    c, dy = inputs(10, 3, size, "gate", dtype)
    dim = 3 * size
    wide = torch.zeros(10, 3 * dim + 5, dtype=dtype)
    for k, t in enumerate((c["x"], c["z"], dy)):
        wide[:, k * dim + 1:(k + 1) * dim + 1] = t
    on = up(wide)
    v = [on[:, k * dim + 1:(k + 1) * dim + 1] for k in range(3)]
    a = dict(groups=3, act="gate")
    w, b = up(c["weight"]), up(c["bias"])
    y = m3.mamba3_groupnorm_fwd(up(c["x"]), w, b, z=up(c["z"]), **a)
    room = torch.full((10 * dim + 2,), 7.0, dtype=dtype, device=device())
    out = m3.mamba3_groupnorm_fwd(v[0], w, b, z=v[1], y=room[1:-1].view(10, dim), **a)
    assert torch.equal(out, y) and float(room[0]) == 7 and float(room[-1]) == 7
    g = m3.mamba3_groupnorm_bwd(up(c["x"]), w, b, z=up(c["z"]), dy=up(dy), **a)
    h = m3.mamba3_groupnorm_bwd(v[0], w, b, z=v[1], dy=v[2], **a)
    for k in g:
        assert R.off(h[k], (g[k].cpu().double(), g[k].cpu().double().abs() * 4)) <= 1, k
    # more dimensions than two
    three = m3.mamba3_groupnorm_fwd(up(c["x"]).view(2, 5, dim), w, b, z=up(c["z"]).view(2, 5, dim), **a)
    assert three.shape == (2, 5, dim) and torch.equal(three.view(10, dim), y)


def test_no_rows():
    x = torch.empty(0, 64, device=device())
    w = torch.ones(64, device=device())
    assert m3.mamba3_groupnorm_fwd(x, w, groups=4).shape == (0, 64)
    g = m3.mamba3_groupnorm_bwd(x, w, w, dy=x, groups=4)
    assert not g["dweight"].any() and not g["dbias"].any()
