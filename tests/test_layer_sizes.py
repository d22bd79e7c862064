"""The sizes that the layer operators take and refuse: the bound is on the workgroups that a call's launches
have, by the header's formulas. On the CPU; no compute call is made."""
import ctypes

import pytest

import state_space_sequence_mamba3_amd as m3
from tests.test_layer_abi import EINVAL, NAMES, OK, conv, conv_bwd, conv_step, scan, scan_bwd, step
from tests.test_layer_abi import lib  # noqa: F401  (a fixture)


def apart(i):
    """Addresses 2^42 bytes apart: no two arrays of a call overlap, whatever its sizes."""
    return 0x1000000000000 + i * (1 << 42)


def ceil(a, b):
    return -(-a // b)


MOST = (1 << 24) - 1
F32, BF16 = m3.MAMBA3_F32, m3.MAMBA3_BF16
SCAN_C = {4: (256, 256), 8: (128, 128), 16: (64, 64), 32: (64, 32), 64: (32, 16), 128: (16, 16)}


@pytest.mark.parametrize("make,over,want", [
    # refused when the bound counted 16 channels a workgroup, and the backward's sums for the forward too
    (scan, dict(batch=1, seqlen=1 << 20, dim=1 << 14, dstate=16, ngroups=1), OK),
    (scan_bwd, dict(fwd_batch=1, fwd_seqlen=1 << 20, fwd_dim=1 << 14, fwd_dstate=16, fwd_ngroups=1), OK),
    (scan, dict(batch=1, seqlen=1 << 30, dim=64, dstate=128, ngroups=1), OK),
    (scan, dict(batch=1 << 18, seqlen=1, dim=1 << 12, dstate=16, ngroups=1), EINVAL),        # 2^18 * 64 workgroups
    (scan, dict(batch=(1 << 18) - 1, seqlen=1, dim=1 << 12, dstate=16, ngroups=1), OK),
    (scan_bwd, dict(fwd_batch=1, fwd_seqlen=1 << 30, fwd_dim=64, fwd_dstate=128, fwd_ngroups=1), EINVAL),
    (conv, dict(batch=1, seqlen=1 << 20, dim=1 << 16), OK),
    (conv, dict(batch=1, seqlen=1 << 30, dim=512, conv_out=None), EINVAL),                   # 2^24 workgroups
    (conv, dict(batch=1, seqlen=(1 << 30) - 7 * 64, dim=512), OK),                           # and 6 of the state's
    (conv, dict(batch=1, seqlen=(1 << 30) - 6 * 64, dim=512), EINVAL),
    (conv, dict(batch=1, seqlen=1 << 30, dim=1), EINVAL),
    (conv_bwd, dict(fwd_batch=1, fwd_seqlen=1 << 30, fwd_dim=256), OK),
    (conv_bwd, dict(fwd_batch=1, fwd_seqlen=1 << 30, fwd_dim=257), EINVAL),                  # 2^23 * 2
    (conv_step, dict(batch=1 << 20, dim=1 << 14), EINVAL), (conv_step, dict(batch=(1 << 20) - 1, dim=1 << 14), OK),
    (conv_step, dict(batch=1 << 18, dim=(1 << 14) - 1), EINVAL), (conv_step, dict(batch=(1 << 18) - 1, dim=(1 << 14) - 1), OK),
    (step, dict(batch=1 << 18, dim=1 << 12, dstate=32), EINVAL), (step, dict(batch=(1 << 18) - 1, dim=1 << 12, dstate=32), OK),
])
def test_bounds(lib, make, over, want):  # noqa: F811
    check(lib, make(**over), want)


def check(lib, a, want):  # noqa: F811
    n, inner = 0, getattr(a, "fwd", None)
    for s in (inner, a) if inner is not None else (a,):
        for f, t in s._fields_:
            if t is ctypes.c_void_p and getattr(s, f):
                n += 1
                setattr(s, f, apart(n))
    if hasattr(a, "workspace_bytes"):
        a.workspace_bytes = 1 << 41
    assert getattr(lib, f"mamba3_{NAMES[type(a)]}_validate")(ctypes.byref(a)) == want


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_documented_workgroups(lib, dtype):  # noqa: F811
    """The header's formulas decide, at the last size taken and the first refused."""
    es = 2 if dtype == BF16 else 4
    for dim in (1, 3, 4, 7, 8, 100, 256, 300, 512, 5000):
        v = 16 // es
        c = 64 * (v if dim >= v else 1)
        t = MOST // ceil(dim, c) * 64       # tokens; without sequences there is no state to count
        for back, tok, c in ((False, 64, c), (True, 128, 256 if dim >= 4 else 64)):
            t = min(MOST // ceil(dim, c) * tok - tok * (ceil(3 * dim, 256) + 1), (1 << 30) - tok)
            count = lambda T: ceil(T, tok) * ceil(dim, c) + ceil(3 * dim, 256)   # noqa: E731, B023
            for T in (t, t + tok * (2 * ceil(3 * dim, 256) + 4)):
                if T > 1 << 30:
                    continue
                a = conv_bwd(fwd_batch=1, fwd_seqlen=T, fwd_dim=dim, fwd_dtype=dtype) if back else \
                    conv(batch=1, seqlen=T, dim=dim, dtype=dtype)
                check(lib, a, OK if count(T) <= MOST else EINVAL)
    for top, (fwd, bwd) in SCAN_C.items():
        for n in (top, top // 2 + 1):
            for dim, g in ((2048, 2), (100, 1), (6, 3)):
                per = g * ceil(dim // g, fwd)
                for b in (MOST // per, MOST // per + 1):
                    check(lib, scan(batch=b, seqlen=1, dim=dim, dstate=n, ngroups=g, dtype=dtype), OK if b * per <= MOST else EINVAL)
                per = g * ceil(dim // g, bwd)
                for b in (MOST // per, MOST // per + 1):
                    need = max(b * per, ceil(2 * b * g * n, 256) + ceil(dim * (n + 2), 256))
                    check(lib, scan_bwd(fwd_batch=b, fwd_seqlen=1, fwd_dim=dim, fwd_dstate=n, fwd_ngroups=g, fwd_dtype=dtype),
                          OK if need <= MOST else EINVAL)
                per = ceil(dim, fwd)
                for b in (MOST // per, MOST // per + 1):
                    check(lib, step(batch=b, dim=dim, dstate=n, ngroups=g, dtype=dtype), OK if b * per <= MOST else EINVAL)
