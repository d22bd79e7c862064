"""The selective scan over sequences of many segments, held to bounds that run through its recurrence
(tests/layer_bounds.py)."""
import ctypes
import math

import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_bounds as LB
from tests.gpu_util import note
from tests.test_gpu_layer import BF16, F32, up

pytestmark = pytest.mark.gpu


def pad256(n):
    return -(-n // 256) * 256


def segment_bytes(rows, dim, N, S, packed):
    return pad256(rows * dim * N * 4) + pad256(rows * dim * 4) + (pad256(rows * 16) + pad256((S + 1) * 4) if packed else 0)


def assert_segments(case, seg):
    """The workspaces are those of segments of `seg` tokens: the test would otherwise stop covering them."""
    b, L, dim, N, G, cu = case
    S, T = (len(cu) - 1 if cu else b), b * L
    rows = S + math.ceil(T / seg) if cu else S * math.ceil(L / seg)
    a = m3.SelectiveScanArgs(batch=b, seqlen=L, dim=dim, dstate=N, ngroups=G, dtype=m3.MAMBA3_F32, cu_seqlens=256 if cu else None,
                             nseq=S if cu else 0)
    seg_b = segment_bytes(rows, dim, N, S, bool(cu))
    assert m3.lib().mamba3_selective_scan_workspace_size(ctypes.byref(a)) == seg_b
    # the backward's: the segments', their gradients, the stored states and sums of steps, dB and dC, dA, dD and ddt_bias
    npl, lpc = (4, 1 if N <= 4 else 2 if N <= 8 else 4 if N <= 16 else 8 if N <= 32 else 16) if N <= 64 else (8, 16)
    per, stored = G * math.ceil(dim // G / (256 // lpc)), T // 8 + rows
    want = seg_b + pad256(rows * dim * N * 4) + pad256(stored * per * 256 * npl * 4) + pad256(stored * per * (256 // lpc) * 4) + \
        pad256(per * T * 2 * N * 4) + pad256(rows * dim * N * 4) + pad256(rows * 2 * dim * 4)
    q = m3.SelectiveScanBwdArgs(fwd=a)
    assert m3.lib().mamba3_selective_scan_bwd_workspace_size(ctypes.byref(q)) == want


SEGMENTS = [  # one sequence of 9, 10, 16, 17 and 18 segments of 64 tokens: the chain takes eight at a time
    (1, 576, 8, 16, 1, None), (1, 577, 8, 16, 1, None), (1, 1024, 8, 16, 1, None), (1, 1025, 8, 16, 1, None),
    (1, 1100, 9, 16, 1, None), (2, 600, 12, 24, 3, None), (1, 700, 6, 3, 2, None), (1, 640, 6, 64, 1, None), (1, 600, 5, 128, 1, None),
    # packed: 10, none, 9, 1 and 18 segments; the sequences' first segments in the table's order
    (1, 2402, 8, 16, 1, [0, 577, 577, 1153, 1160, 2300]), (1, 1300, 7, 7, 1, [0, 3, 1100, 1300]), (1, 1201, 10, 40, 2, [0, 600, 1201])]


@pytest.mark.parametrize("dtype,positive,plain", [(F32, True, False), (F32, False, True), (BF16, True, False)])
@pytest.mark.parametrize("case", SEGMENTS)
def test_scan_of_many_segments(case, dtype, positive, plain):
    note(f"segments {case} {dtype} positive={positive} plain={plain}")
    assert_segments(case, 64)
    c = LB.scan_case(*case, 17 + case[1], positive, dtype, plain)
    last = case[5][-1] if case[5] else case[1]      # tokens behind the last sequence take no part
    want = LB.scan(**c, window=64)
    args = [up(c[k]) for k in ("x", "dt", "A", "B", "C", "D")]
    kw = dict(z=up(c["z"]), dt_bias=up(c["bias"]), dt_softplus=c["softplus"], h_in=up(c["h_in"]),
              cu_seqlens=up(torch.tensor(case[5], dtype=torch.int32)) if case[5] else None)
    y, h = m3.mamba3_selective_scan_fwd(*args, **kw)
    got = m3.mamba3_selective_scan_bwd(*args, **kw, dy=up(c["dy"]), dh_out=up(c["dh_out"]))
    got.update(y=y, h_out=h)
    for k, t in got.items():
        if k in ("y", "dx", "ddt", "dz", "dB", "dC"):
            t, want[k] = t[:, :last], tuple(w[:, :last] for w in want[k])
        assert bool(torch.isfinite(t).all()), k
        assert LB.off(t, want[k]) <= 1, (k, LB.off(t, want[k]))
        note(f"  {k} {LB.off(t, want[k]):.3f}")
