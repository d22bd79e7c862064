"""Calls of the gated scan whose launches are as large as the header allows: 2^32 threads and more in parts."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu

PART = 1 << 20


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,L,D", [((1 << 22) + 3, 1, 2), ((1 << 23) + 5, 1, 1), ((1 << 21) + 1, 2, 130)])
def test_many_sequences(b, L, D, dtype):
    """Many short sequences have what they have in smaller batches, bit for bit."""
    note(f"gated scan of {b} sequences of {L} x {D} {dtype}")
    g = torch.Generator(device=device()).manual_seed(b)
    x, gate, dy = (torch.randn((b, L, D), generator=g, device=device(), dtype=dtype) for _ in range(3))
    h, dh = (torch.randn((b, D), generator=g, device=device()) for _ in range(2))
    w = torch.rand(D, generator=g, device=device())
    a = dict(form="forget", i=x)
    y, out = m3.mamba3_gated_scan_fwd(x, gate, w, h_in=h, **a)
    got = dict(y=y, h_out=out, **m3.mamba3_gated_scan_bwd(x, gate, w, dy=dy, dh_out=dh, h_in=h, **a))
    for k in range(0, b, PART):
        s = slice(k, min(k + PART, b))
        p = dict(form="forget", i=x[s])
        y, out = m3.mamba3_gated_scan_fwd(x[s], gate[s], w, h_in=h[s], **p)
        want = dict(y=y, h_out=out, **m3.mamba3_gated_scan_bwd(x[s], gate[s], w, dy=dy[s], dh_out=dh[s], h_in=h[s], **p))
        del want["dweight"]                     # (summed over other rows)
        for n in want:
            assert torch.equal(got[n][s], want[n]), (n, k)


def test_weights_of_many_sequences():
    """dweight has every row's share: all gradients but those of a few sequences, the first and the last among them, are
    zero, which adds nothing."""
    b, D = (1 << 23) + 5, 3
    note(f"gated scan, weights of {b} sequences")
    g = torch.Generator().manual_seed(1)
    at = torch.cat([torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, b - 1]), torch.randint(b, (40,), generator=g)]).unique()
    few = {k: torch.randn((len(at), 1, D), generator=g) for k in ("x", "gate", "dy")}
    h, w = torch.randn((len(at), D), generator=g), torch.randn(D, generator=g) - 4
    ref = R.scan(few["x"], few["gate"], w, "decay", 8.0, None, None, h, None, few["dy"])["dweight"]
    on = at.to(device())
    wide = {k: torch.zeros((b, 1, D), device=device()) for k in few}
    for k in few:
        wide[k][on] = few[k].to(device())
    hin = torch.zeros((b, D), device=device())
    hin[on] = h.to(device())
    got = m3.mamba3_gated_scan_bwd(wide["x"], wide["gate"], w.to(device()), dy=wide["dy"], h_in=hin)
    assert R.off(got["dweight"], ref) <= 1
