"""Which way the gated scan takes for a call, seen in its workspace: whole sequences need none, segments and the one
pass lay out their own. On the CPU, from the sizes alone."""
import ctypes

import pytest

import state_space_sequence_mamba3_amd as m3
from tests.test_gated_abi import BF16, F32, ceil, fake, scan, scan_bwd
from tests.test_layer_abi import lib  # noqa: F401  (a fixture)

# batch, seqlen, dim, sequences packed, tokens of a segment: segments of more than 64 packed sequences (their rows in a
# table) that rows join by themselves and that the chain joins; the chain over up to 64 packed sequences, whose rows are
# counted, and over a padded batch
PLANS = {"table": (1, 1500, 40, 100, 32), "table and chain": (1, 8300, 40, 100, 128), "counted and chain": (1, 8300, 40, 5, 128),
         "chain": (1, 9000, 12, 0, 128)}


def al256(n):
    return ceil(n, 256) * 256


def packed(nseq):
    return dict(cu_seqlens=fake(20), nseq=nseq) if nseq else {}


def size(lib, a):  # noqa: F811
    return getattr(lib, f"mamba3_gated_scan{'_bwd' if isinstance(a, m3.GatedScanBwdArgs) else ''}_workspace_size")(ctypes.byref(a))


def run_bytes(b, L, D, nseq, tokens, arrays, channel):
    rows = nseq + ceil(L, tokens) if nseq else b * ceil(L, tokens)
    table = al256(16 * rows) + al256(4 * (nseq + 1)) if nseq > 64 else 0
    return arrays * al256(4 * rows * D) + (al256(4 * D) if channel else 0) + table


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("plan", PLANS)
def test_segments(lib, plan, dtype):  # noqa: F811
    b, L, D, nseq, tokens = PLANS[plan]
    assert (ceil(L, tokens) > 64) == ("chain" in plan)
    assert size(lib, scan(batch=b, seqlen=L, dim=D, dtype=dtype, **packed(nseq))) == run_bytes(b, L, D, nseq, tokens, 2, False)
    a = scan_bwd(fwd_batch=b, fwd_seqlen=L, fwd_dim=D, fwd_dtype=dtype, **{"fwd_" + k: v for k, v in packed(nseq).items()})
    assert size(lib, a) == run_bytes(b, L, D, nseq, 32, 4, True) and ceil(L, 32) > 32       # (the backward's chain)


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


@pytest.mark.parametrize("dim", [255, 127, 257])
def test_workgroups_of_odd_counts(lib, dim):  # noqa: F811
    """128 channels a workgroup with odd counts too, but 64 where the count is one above a multiple of 128."""
    from tests.test_gated_abi import EINVAL, MOST, OK, apart
    tiles = ceil(dim, 64 if dim % 128 == 1 else 128)
    for b in (MOST // tiles, MOST // tiles + 1):
        apart(lib, scan(batch=b, seqlen=2, dim=dim), OK if b * tiles <= MOST else EINVAL)
