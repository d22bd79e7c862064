"""The decay form of the gated recurrence with weights that are not finite or far out: the scan whole, in segments,
packed and in one pass, its backward, and the step."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_gated import BF16, F32, call, inputs, up

pytestmark = pytest.mark.gpu

# whole sequences, two that are joined by their own rows, packed ones, an odd count of channels, one pass
CASES = [(2, 37, 64, None), (1, 1000, 12, None), (1, 700, 20, [0, 64, 65, 300, 700]), (3, 40, 13, None), (1, 1200, 4096, None)]
HIT = [2, 5, 11]


def all_of(c, back):
    return {**call(c), **call(c, back)}


def step_of(c):
    w, h = up(c["weight"]), up(c["h_in"])[:c["x"].shape[0]].clone()
    t = {k: up(c[k][:, 0].contiguous()) for k in ("x", "gate", "i", "z")}
    y = m3.mamba3_gated_step(t["x"], t["gate"], w, h=h, i=t["i"], z=t["z"])
    return dict(y=y, h=h)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_nan_weights_show(case, dtype):
    """A weight that is NaN makes everything of its channel NaN, and nothing of another."""
    note(f"NaN weights {case} {dtype}")
    c, back = inputs(*case, "decay", dtype, True, True, True)
    clean = [all_of(c, back), step_of(c)]
    c["weight"][HIT] = float("nan")
    keep = torch.ones(case[2], dtype=torch.bool)
    keep[HIT] = False
    for got, want in zip([all_of(c, back), step_of(c)], clean):
        for k in got:
            assert bool(got[k][..., HIT].isnan().all()), k
            assert torch.equal(got[k][..., keep], want[k][..., keep]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES[:4])
def test_weights_far_below(case, dtype):
    """softplus(w) is zero: a = 1 and u = 0, the state stays and no gradient reaches input, gates and weight."""
    note(f"weights far below {case} {dtype}")
    c, back = inputs(*case, "decay", dtype, True, True, True)
    far = torch.tensor([float("-inf"), -3.3e38, -2.5e38])
    c["weight"][HIT] = -200.0
    ref = R.scan(**c, **back)                   # (a softplus of 1e-87, whose u counts as zero)
    c["weight"][HIT] = far
    got = all_of(c, back)
    for k in got:
        assert R.off(got[k], ref[k]) <= 1, k
    assert torch.equal(got["h_out"].cpu()[:, HIT], c["h_in"][:, HIT])
    for k in ("dx", "dgate", "di", "dweight"):
        assert not got[k][..., HIT].any(), k
    assert torch.equal(step_of(c)["h"].cpu()[:, HIT], c["h_in"][:case[0], HIT])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES[:4])
@pytest.mark.parametrize("rate", [8.0, 3e38])
def test_weights_far_above(case, rate, dtype):
    """rate softplus(w) leaves fp32's range: a = 0 and u = 1, a state is its own token's, and no gradient reaches gate and
    weight."""
    note(f"weights far above {case} {dtype} rate {rate}")
    c, back = inputs(*case, "decay", dtype, True, True, True)
    c["rate"] = rate
    c["weight"][HIT] = 1e30
    if rate > 8:
        c["weight"][:] = 10.0                   # (every channel's decay is zero)
    ref = R.scan(**c, **back)
    if rate == 8:
        c["weight"][HIT] = torch.tensor([1e38, 3e38, float("inf")])
    got = all_of(c, back)
    for k in got:
        assert R.off(got[k], ref[k]) <= 1, k
    for k in ("dgate", "dweight", "dh_in"):
        assert not got[k][..., HIT].any(), k
    assert bool(step_of(c)["h"].isfinite().all())
