"""The norms where squares or differences are at the ends of what fp32 holds: rows of small values whose squares, scaled up,
add up past the range; centered groups of equal values far from zero."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests import layer_bounds as LB
from tests import layer_ref as LR
from tests.gpu_util import note
from tests.test_gpu_groupnorm import BF16, F32, check, inputs, rand, up

pytestmark = pytest.mark.gpu

# mean squares of 2^-98 to 2^-79, and those of values next to the least normal ones
SMALL = [1.2e-15, 2.5e-15, 2e-14, 1.5e-13, 4e-13, 9e-13, 1.3e-12, 1e-36]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("size", [64, 511, 600, 2000, 4096, 8192])
def test_small_groups(size, center, dtype):
    """Groups of small values with eps 0: their norm has the size of one, however many they are."""
    note(f"group norm small values size {size} center {center} {dtype}")
    groups = len(SMALL) if size * len(SMALL) <= 8192 * 8 else 4
    c, dy = inputs(5, groups, size, "none", dtype, mean=0.0)
    for k in range(groups):
        c["x"].view(5, groups, size)[:, k] *= SMALL[k]
    check(c, dy, groups, "none", center, 0.0)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("dim", [512, 1024, 2048, 4096, 8192, 8200, 1 << 17])
def test_small_rows(dim, types):
    """The same of the RMS norm's rows, forward and backward."""
    note(f"rms norm small values {dim} {types}")
    dtype, rt = types
    g = torch.Generator().manual_seed(dim)
    rows = len(SMALL) - 1                   # (not the least: its gradient leaves the range)
    s = (rand(g, rows, dim).double() * torch.tensor(SMALL[:rows]).double()[:, None]).to(rt)
    w, dy = rand(g, dim) * 0.1 + 1, rand(g, rows, dim, dtype=dtype)
    _, v = LR.norm(s, None, w, 0.0)
    got = m3.mamba3_rmsnorm_fwd(up(s).to(dtype), up(w), eps=0.0)
    LR.check(got["y"], v, v, LB.norm_count(dim), "y")
    ref, mag = LR.norm_bwd(s, w, dy, None, 0.0), LR.norm_bwd(s, w, dy, None, 0.0, mag=True)
    got = m3.mamba3_rmsnorm_bwd(up(s), up(w), dy=up(dy), eps=0.0)
    LR.check(got["dx"], ref[0], mag[0], LB.norm_bwd_count(dim), "dx")
    LR.check(got["dweight"], ref[1], mag[1], LB.dweight_count(rows, dim), "dweight")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("eps", [1e-5, 1e-26, 1e-30])
@pytest.mark.parametrize("act", ["none", "gate"])
@pytest.mark.parametrize("size", [24, 100, 600, 5000])
def test_equal_values_far_from_zero(size, act, eps, dtype):
    """A centered group of equal values is its bias, wherever it lies: what the rounding of its mean leaves is no
    deviation. Its gradient is that of a group of zeros."""
    note(f"group norm equal values size {size} {act} eps {eps} {dtype}")
    far = [1e3, 1e6, 3e8, 1e9, -3.3e9, 1e12, 1e20, -1.7e30, 3e38]
    rows, groups = 6, len(far)
    c, dy = inputs(rows, groups, size, act, dtype)
    x = c["x"].view(rows, groups, size)
    x[::2] = 0.0
    ref = R.groupnorm(c["x"], c["weight"], c["bias"], groups, c["z"], act, True, eps, dy)
    x[::2] = torch.tensor(far, dtype=dtype)[:, None]
    a = dict(groups=groups, z=up(c["z"]), act=act, eps=eps)
    got = dict(y=m3.mamba3_groupnorm_fwd(up(c["x"]), up(c["weight"]), up(c["bias"]), **a),
               **m3.mamba3_groupnorm_bwd(up(c["x"]), up(c["weight"]), up(c["bias"]), dy=up(dy), **a))
    # The differences that are summed at last are equal and within the deviation (their mean's square is at most the
    # variance with eps), and their mean is off by DEPTH + 4 roundings of them: so much n is off, in deviations.
    # That mean's square is taken off the squares' mean with as many roundings, twice, halved by the root.
    n, r = R.DEPTH + 4, eps ** -0.5
    sh = lambda t: t.double().view(rows, groups, size)   # noqa: E731
    sz = dsz = torch.ones(rows, groups, size).double()
    if act == "gate":
        sz, _, dsz, _ = R.silu(sh(c["z"]))
    w, d = c["weight"].double().view(groups, size).abs(), sh(dy) * sz
    more = dict(y=n * w * sz.abs(), dz=n * w * (sh(dy) * dsz).abs(), dbias=0 * w, dweight=n * d[::2].abs().sum(0))
    dn = (d * w).abs()
    more["dx"] = (2 * n + 1) * r * (dn + dn.mean(-1, keepdim=True))
    for k in got:
        v, e = ref[k]
        extra = more[k].clone()
        if extra.dim() == 3:
            extra[1::2] = 0
        assert not got[k].isnan().any(), k
        assert R.off(got[k], (v, e + extra.reshape(e.shape))) <= 1, k


@pytest.mark.parametrize("size", [100, 600, 5000])
def test_neighbours_far_from_zero(size):
    """Groups of two neighbouring fp32 values keep their deviations, which are below what the mean's rounding leaves."""
    note(f"group norm neighbours size {size}")
    g = torch.Generator().manual_seed(size)
    far = torch.tensor([1e3, -1e6, 1.1e9, 1e20, -1.7e30])
    rows, groups = 6, len(far)
    x = far[:, None].expand(groups, size).repeat(rows, 1, 1)
    up_ = torch.rand(x.shape, generator=g) < torch.tensor([0.5, 0.2, 0.05, 0.5, 0.3, 0.1]).view(rows, 1, 1)
    up_[..., 3] = True
    x = torch.where(up_, torch.nextafter(x, torch.tensor(float("inf"))), x)
    d = x.double() - far.double()[:, None]                  # (exact; the mean of so small numbers loses nothing in 64 bits)
    d = d - d.mean(-1, keepdim=True)
    n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-30)
    y = m3.mamba3_groupnorm_fwd(up(x.reshape(rows, -1)), groups=groups, eps=1e-30).view(n.shape)
    # differences of neighbours are exact; their mean, within the deviation, is off by DEPTH + 4 roundings of it; three
    # more of n itself, and its deviation's: the squares' sum, root and what is taken off it
    c = R.DEPTH + 4
    assert R.off(y, (n, c + n.abs() * (3 + (R.DEPTH + 6) / 2 + 4 + c))) <= 1
