"""Layer operators at sizes whose arrays pass 2^31 elements."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_layer import BF16, gen, rand, up

pytestmark = pytest.mark.gpu


def test_selective_scan_of_a_long_sequence():
    """More than 2^31 values of B and of C: the first tokens, and the last ones of a state that has forgotten what
    lies 300 tokens back (decays of e^-0.3 a token at least), equal the 64-bit form."""
    L, D, N, n = (1 << 25) + 77, 4, 64, 200
    note(f"scan of {L} tokens, B and C {L * N * 2 >> 20} MiB each")
    g = torch.Generator(device=device()).manual_seed(3)
    x, dt = (torch.randn((1, L, D), generator=g, device=device(), dtype=BF16) for _ in range(2))
    B, C = (torch.randn((1, L, 1, N), generator=g, device=device(), dtype=BF16) for _ in range(2))
    A, skip, bias = -1 - rand(gen(1), D, N).abs(), rand(gen(2), D), torch.full((D,), 3.0)
    y, h = m3.mamba3_selective_scan_fwd(x, dt.clamp(min=-3.5), up(A), B, C, up(skip), dt_bias=up(bias), dt_softplus=True)
    for a, lo, hi in ((0, 0, n), (L - 300 - n, L - n, L)):
        part = [t[:, a:hi].cpu() for t in (x, dt.clamp(min=-3.5), B, C)]
        ref, mag = (R.scan(part[0], part[1], A, part[2], part[3], skip, None, bias, True, None, None, mag=m) for m in (False, True))
        # as in the operator's own tests, 500 tokens; what came before is e^-90 of it
        R.check(y[:, lo:hi], ref["y"][:, lo - a:], mag["y"][:, lo - a:], 70 * 500 + N + 32, f"y {lo}")
    R.check(h, ref["h_out"], mag["h_out"], 70 * 500 + 16, "h_out")
