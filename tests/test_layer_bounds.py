"""The close bounds of the layer operators' tests on the CPU: their values are the plain references', and a mistake
as small as one rounding to bf16, planted in the 64-bit form, lies outside them."""
import pytest
import torch

from tests import layer_bounds as LB
from tests import layer_ref as R

CASES = [(1, 300, 8, 16, 1, None), (1, 577, 8, 16, 1, None), (1, 1100, 8, 16, 1, [0, 577, 577, 1099, 1100]),
         (2, 300, 12, 24, 3, None)]


def bf16(v):
    return v.bfloat16().double()


@pytest.mark.parametrize("positive", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_scan_values(case, positive):
    for plain in (True, False):
        c = LB.scan_case(*case, 5, positive, plain=plain)
        w = LB.scan(**c, window=64)
        ref = R.scan(*[c[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "bias", "softplus", "h_in", "cu", "dy", "dh_out")])
        for k, (v, e) in w.items():
            if k != "dz" or not plain:
                assert float((v - ref[k]).abs().max()) <= 1e-12 * float(ref[k].abs().max()), k
            assert bool((e >= 0).all()) and bool(torch.isfinite(e).all()), k
        # the rounded references themselves are inside
        assert all(LB.off(v.float(), (v, e)) <= 1 for v, e in w.values())


@pytest.mark.parametrize("positive", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_a_rounded_state_is_seen(case, positive):
    """The state that enters the fourth segment, or the gradient that leaves it, rounded to bf16 once."""
    c = LB.scan_case(*case, 5, positive)
    w = LB.scan(**c, window=64)
    for which, at, seen in (("h", 192, ("y", "dC", "dz")), ("g", 191, ("dx", "dB", "dh_in"))):
        bad = LB.scan(**c, window=64, spoil=lambda what, t, v: bf16(v) if (what, t) == (which, at) else v)   # noqa: B023
        for k in seen:
            assert LB.off(bad[k][0].float(), w[k]) > 2, (which, k)


def test_a_lost_segment_is_seen():
    """A state or gradient that a later group of segments takes up as zero, or one segment too early."""
    c = LB.scan_case(1, 1100, 8, 16, 1, None, 6, True)
    w = LB.scan(**c, window=64)
    for which, at, seen in (("h", 512, ("y", "dC", "ddt")), ("h", 1024, ("y", "h_out")), ("g", 587, ("dx", "dB")),
                            ("g", 75, ("dx", "dh_in"))):
        bad = LB.scan(**c, window=64, spoil=lambda what, t, v: v * 0 if (what, t) == (which, at) else v)   # noqa: B023
        assert all(LB.off(bad[k][0].float(), w[k]) > 100 for k in seen), (which, at)


@pytest.mark.parametrize("dim", [513, 2049, 8192, 8201])
def test_a_rounded_statistic_is_seen(dim):
    """1 / rms rounded to bf16, forwards and backwards."""
    g = torch.Generator().manual_seed(dim)
    s, w, dy = torch.randn(8, dim, generator=g), torch.randn(dim, generator=g) + 1, torch.randn(8, dim, generator=g)
    r = 1 / torch.sqrt((s.double() ** 2).mean(-1, keepdim=True) + 1e-5)
    _, v = R.norm(s, None, w, 1e-5)
    ref, mag = R.norm_bwd(s, w, dy, None, 1e-5), R.norm_bwd(s, w, dy, None, 1e-5, mag=True)

    def gradients(r):
        sh, wd = s.double() * r, dy.double() * w
        return r * (wd - sh * (wd * sh).mean(-1, keepdim=True)), (dy.double() * sh).sum(0)

    for rounded in (False, True):
        q = bf16(r) if rounded else r
        ds, dw = gradients(q)
        results = ((s.double() * q * w, v, v, LB.norm_count(dim)), (ds, ref[0], mag[0], LB.norm_bwd_count(dim)),
                   (dw, ref[1], mag[1], LB.dweight_count(8, dim)))
        for got, want, m, count in results:
            if rounded:
                with pytest.raises(AssertionError):
                    R.check(got.float(), want, m, count, "planted")
            else:
                R.check(got.float(), want, m, count, "sound")
