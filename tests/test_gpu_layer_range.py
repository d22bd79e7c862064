"""The layer operators on values at the ends of fp32's range, where a formula's intermediate results leave
the range that its inputs and outputs keep."""
import ctypes

import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_bounds as LB
from tests import layer_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_layer import BF16, F32, gen, rand, up

pytestmark = pytest.mark.gpu

# one wave a row, four, eight and sixteen, rows that are read again; aligned and not; more rows than workgroups
ROWS = [(9, 64), (2600, 65), (11, 1000), (2300, 1024), (1100, 2048), (5, 2049), (600, 4096), (3, 8191), (300, 8192),
        (5, 8200), (1100, 8201)]


def scaled_rows(g, rows, dim, dtype, scales):
    """Rows whose values are of one size each, taken from `scales` in turn."""
    s = torch.tensor([scales[i % len(scales)] for i in range(rows)]).double()
    return (rand(g, rows, dim).double() * s[:, None]).to(dtype)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("rows,dim", ROWS)
def test_rmsnorm_of_tiny_and_huge_rows(rows, dim, eps, types):
    """The norm of a finite row is finite, whether or not its squares are."""
    note(f"rmsnorm range {rows}x{dim} eps {eps} {types}")
    dtype, rt = types
    g = gen(rows + dim)
    x = scaled_rows(g, rows, dim, dtype, (1.0, 1e-20, 1e20, 1e-30, 1e15, 1e30, 1e-15, 1e-36, 1e36))
    res, w = (x.double() * 0.25).to(rt), rand(g, dim) * 0.1 + 1
    s, v = R.norm(x, res, w, eps)
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual=up(res), eps=eps)
    R.check(got["y"], v, v, LB.norm_count(dim), "y")
    R.check(got["residual"], s, s, 1, "residual")


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("rows,dim", ROWS)
def test_rmsnorm_bwd_of_tiny_and_huge_rows(rows, dim, eps, types):
    note(f"rmsnorm backward range {rows}x{dim} eps {eps} {types}")
    dtype, rt = types
    g = gen(rows + dim + 1)
    s = scaled_rows(g, rows, dim, rt, (1.0, 1e-20, 1e20, 1e-25, 1e15, 1e25, 1e-15))
    dy, w = rand(g, rows, dim, dtype=dtype), rand(g, dim) * 0.1 + 1
    for dres in (None, rand(g, rows, dim, dtype=rt)):
        ref, mag = R.norm_bwd(s, w, dy, dres, eps), R.norm_bwd(s, w, dy, dres, eps, mag=True)
        got = m3.mamba3_rmsnorm_bwd(up(s), up(w), dy=up(dy), dresidual_out=up(dres), eps=eps)
        for k in ("dx", "dresidual"):
            R.check(got[k], ref[0], mag[0], LB.norm_bwd_count(dim), k)
        R.check(got["dweight"], ref[1], mag[1], LB.dweight_count(rows, dim), "dweight")
    # dresidual in dresidual_out's place
    own, keep, dw = up(dres), [up(t) for t in (s, dy, w)], torch.empty(dim, device=device())
    code = {F32: m3.MAMBA3_F32, BF16: m3.MAMBA3_BF16}
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=device())
    a = m3.RmsnormBwdArgs(rows, dim, code[dtype], code[rt], eps, 0, keep[0].data_ptr(), keep[1].data_ptr(), own.data_ptr(),
                          keep[2].data_ptr(), None, own.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel())
    assert m3.lib().mamba3_rmsnorm_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == m3.MAMBA3_OK
    torch.cuda.synchronize()
    assert torch.equal(own, got["dresidual"]) and torch.equal(dw, got["dweight"])


def test_rmsnorm_of_rows_without_a_norm():
    """Zeros with eps 0 have no norm, with eps a norm of zeros; infinite and NaN rows stay by themselves."""
    x = torch.ones(5, 64)
    x[1], x[2, 5], x[3, 7] = 0, float("inf"), float("nan")
    y = m3.mamba3_rmsnorm_fwd(up(x), eps=0.0)["y"].cpu()
    assert bool((y[[0, 4]] - 1).abs().max() < 1e-6) and bool(torch.isnan(y[[1, 3]]).all())
    assert bool(torch.isnan(y[2, 5])) and int((y[2] == 0).sum()) == 63
    y = m3.mamba3_rmsnorm_fwd(torch.zeros(2, 64, device=device()), eps=1e-5)["y"]
    assert bool((y == 0).all())


# ----------------------------------------------------------------------------- states that grow
def growing(kind, L, D, N, g):
    """Inputs of a scan whose states or gradients grow by more than fp32's range over a segment (64 tokens)
    and yet stay in it: A > 0, or steps below zero."""
    x, dt = torch.zeros(1, L, D), torch.ones(1, L, D)
    A = 1 + 0.5 * torch.rand(D, N, generator=g)
    dy = torch.zeros(1, L, D)
    h, dh = torch.zeros(1, D, N), torch.zeros(1, D, N)
    B, C = (0.5 + torch.rand(1, L, 1, N, generator=g) for _ in range(2))
    if kind == "late inputs":           # zero until 30 tokens before the end; gradients from the first 30 alone
        x[:, L - 30:] = rand(g, 1, 30, D)
        dy[:, :30] = rand(g, 1, 30, D)
    elif kind == "late inputs, steps below zero":
        x[:, L - 30:] = rand(g, 1, 30, D)
        dy[:, :30] = rand(g, 1, 30, D)
        A, dt = -A, -dt
    elif kind == "from a tiny state":   # e^100 times larger after a segment, and decays from there
        h = 1e-30 * (1 + torch.rand(1, D, N, generator=g))
        dt[:, 66:] = -1
        dy[:, 100:140] = 0.5 + torch.rand(1, 40, D, generator=g)
    else:                               # the same for the gradient that enters at the end
        dh = 1e-30 * (1 + torch.rand(1, D, N, generator=g))
        dt[:, :L - 66] = -1
        x[:, L - 140:L - 100] = 0.5 + torch.rand(1, 40, D, generator=g)
    return x, dt, A, B, C, h, dy, dh


@pytest.mark.parametrize("kind,L", [("late inputs", 60), ("late inputs", 400), ("late inputs, steps below zero", 60),
                                    ("late inputs, steps below zero", 400), ("from a tiny state", 400),
                                    ("from a tiny gradient", 400)])
def test_growing_states(kind, L):
    """One sequence, whole (60 tokens) and in segments (400): finite wherever the formula's values are."""
    note(f"growing {kind} {L}")
    D, N = 24, 16
    x, dt, A, B, C, h, dy, dh = growing(kind, L, D, N, gen(L))
    ref, mag = (R.scan(x, dt, A, B, C, None, None, None, False, h, None, dy, dh, mag=m) for m in (False, True))
    assert all(bool((v.abs() < 1e38).all()) for v in ref.values())
    got = dict(zip(("y", "h_out"), m3.mamba3_selective_scan_fwd(up(x), up(dt), up(A), up(B), up(C), h_in=up(h))))
    got.update(m3.mamba3_selective_scan_bwd(up(x), up(dt), up(A), up(B), up(C), dy=up(dy), dh_out=up(dh), h_in=up(h)))
    for k, v in got.items():
        # as in the operator's own tests: a decay is off by 60 roundings of its argument and 10 more a token,
        # for states and gradients both; sums over channels, states and tokens
        R.check(v, ref[k], mag[k], 140 * L + 64 + D + N + L, k)
