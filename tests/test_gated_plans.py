"""Which way the gated scan takes for a call, seen in its workspace: whole sequences need none, segments and the one
pass lay out their own. On the CPU, from the sizes alone."""
import ctypes

import pytest

from tests.test_gated_abi import BF16, F32, ceil, fake, scan
from tests.test_layer_abi import lib  # noqa: F401  (a fixture)


def al256(n):
    return ceil(n, 256) * 256


def packed(nseq):
    return dict(cu_seqlens=fake(20), nseq=nseq) if nseq else {}


def size(lib, a):  # noqa: F811
    return lib.mamba3_gated_scan_workspace_size(ctypes.byref(a))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_pass_has_its_launch(lib, dtype):  # noqa: F811
    """The one pass has 1024 threads a workgroup and takes no call whose workgroups would be 2^32 threads or more."""
    run = 128 if dtype == BF16 else 64

    def pass_bytes(b, L, D):
        rows = b * ceil(L, run)
        return al256(8 * rows * D) + al256(8 * (rows // 8 + b + 1) * D) + 256

    for b, D, tiles in ((255, 5, 1), (1, 8192, 64), (3, 1025, 17)):
        most = ((1 << 22) - 1) // tiles // b                # runs of a sequence
        for n, taken in ((most, True), (most + 1, False), (2 * most, False)):
            if b * n * run <= 1 << 30:
                got = size(lib, scan(batch=b, seqlen=n * run, dim=D, dtype=dtype))
                assert (got == pass_bytes(b, n * run, D)) == taken, (b, n, D)
    # packed: the rows are the runs and one more a sequence
    for nseq, D, tiles in ((1, 8192, 64), (60, 1024, 8)):
        most = ((1 << 22) - 1) // tiles - nseq
        for n, taken in ((most, True), (most + 1, False)):
            if n * run <= 1 << 30:
                rows = nseq + n
                want = al256(8 * rows * D) + al256(8 * (rows // 8 + nseq + 1) * D) + 256
                got = size(lib, scan(batch=1, seqlen=n * run, dim=D, dtype=dtype, **packed(nseq)))
                assert (got == want) == taken, (nseq, n, D)
