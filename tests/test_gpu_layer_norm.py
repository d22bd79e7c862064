"""The RMS norm held to bounds that follow its sums (tests/layer_bounds.py), at row lengths of every arrangement of
waves and with more rows than workgroups."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_bounds as LB
from tests import layer_ref as R
from tests.gpu_util import note
from tests.test_gpu_layer import BF16, F32, norm_inputs, rand, up

pytestmark = pytest.mark.gpu

# aligned and not: one wave a row; four; four with two pieces a lane (eight waves in the backward); with four pieces
# (sixteen); rows that are read again. The larger counts of rows exceed the backward's workgroups.
NORM = [(7, 512), (5000, 512), (4200, 511), (2100, 1023), (300, 1024), (5, 1025), (1100, 2048), (1300, 1999), (3, 2049),
        (5, 3000), (2, 4096), (1100, 4096), (700, 4095), (2, 4097), (600, 8192), (300, 8191), (3, 8193), (1100, 8200), (1100, 8201)]


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,dim", NORM)
def test_rmsnorm(rows, dim, types):
    note(f"rmsnorm {rows}x{dim} {types}")
    dtype, rt = types
    x, res, w, _ = norm_inputs(rows, dim, *types)
    s, v = R.norm(x, res, w, 1e-5)
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual=up(res), eps=1e-5)
    R.check(got["y"], v, v, LB.norm_count(dim), "y")
    R.check(got["residual"], s, s, 1, "residual")
    for carry in (True, False):
        dy, s, w, g = norm_inputs(rows, dim, dtype, rt, seed=7)
        dres = rand(g, rows, dim, dtype=rt) if carry else None
        ref, mag = R.norm_bwd(s, w, dy, dres, 1e-5), R.norm_bwd(s, w, dy, dres, 1e-5, mag=True)
        got = m3.mamba3_rmsnorm_bwd(up(s), up(w), dy=up(dy), dresidual_out=up(dres), eps=1e-5)
        R.check(got["dresidual"], ref[0], mag[0], LB.norm_bwd_count(dim), "dresidual")
        R.check(got["dx"], ref[0], mag[0], LB.norm_bwd_count(dim), "dx")
        R.check(got["dweight"], ref[1], mag[1], LB.dweight_count(rows, dim), "dweight")


@pytest.mark.parametrize("rows,dim", [(4200, 511), (300, 1024), (1100, 2048), (3, 2049), (700, 4095), (1100, 4096), (300, 8191), (2, 8192),
                                      (5, 8201)])
@pytest.mark.parametrize("qblock", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
def test_rmsnorm_quantised(rows, dim, qblock, quant):
    note(f"rmsnorm {quant} {rows}x{dim} block {qblock}")
    x, res, w, _ = norm_inputs(rows, dim, BF16, BF16)
    _, v = R.norm(x, res, w, 1e-5)
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual=up(res), eps=1e-5, quant=quant, qblock=qblock)
    R.check(got["y"], v, v, LB.norm_count(dim), "y")
    block = qblock or dim
    blocks = -(-dim // block)
    pad = torch.nn.functional.pad(v, (0, blocks * block - dim)).view(rows, blocks, block)
    top = 448.0 if quant == "e4m3" else 127.0
    want = pad.abs().amax(-1) / top
    R.check(got["scale"], want, want, LB.norm_count(dim) + 1, "scale")
    ideal = v / got["scale"].cpu().double().repeat_interleave(block, 1)[:, :dim]
    # the nearest 8-bit value of what v is in 32 bits: half a step (2^-4 relative, 2^-10 below 2^-6; 0.5), v's and
    # the quotient's roundings before it
    half = torch.maximum(ideal.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double()) if quant == "e4m3" else torch.tensor(0.5).double()
    err = (LB.norm_count(dim) + 2) * R.U32 * ideal.abs()
    q = got["q"].cpu().double()
    assert bool(((q - ideal).abs() <= half * (1 + 1e-6) + 2 * err).all()) and bool((q.abs() <= top).all())
