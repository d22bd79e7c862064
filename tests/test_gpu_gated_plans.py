"""The gated scan's segments joined by k_gate_chain, and those of more than 64 packed sequences, against the 64-bit form;
h_out in h_in's place."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import note
from tests.test_gated_plans import PLANS
from tests.test_gpu_gated import BF16, F32, call, inputs, up

pytestmark = pytest.mark.gpu


def boundaries(L, nseq):
    """Sequences of all lengths, some of them empty, one much longer than the others."""
    g = torch.Generator().manual_seed(L + nseq)
    cuts = sorted(torch.randint(0, L // 2, (nseq - 4,), generator=g).tolist())
    return [0, 0, *cuts, L - 3, L - 3, L]


@pytest.mark.parametrize("dtype,form,full", [(F32, "decay", False), (BF16, "forget", True), (BF16, "decay", True)])
@pytest.mark.parametrize("plan", PLANS)
def test_plan(plan, dtype, form, full):
    b, L, D, nseq, _ = PLANS[plan]
    note(f"gated scan {plan} {form} {dtype}")
    cu = boundaries(L, nseq) if nseq else None
    assert cu is None or len(cu) == nseq + 1
    c, back = inputs(b, L, D, cu, form, dtype, True, full, True, memory=2.0)
    grads = L < 2000 or (dtype == BF16 and form == "decay")
    ref = R.scan(**c, **(back if grads else {}))
    got = call(c)
    a = {k: up(c[k]) for k in ("x", "gate", "weight", "i", "z")}
    a.update(form=form, cu_seqlens=up(torch.tensor(cu, dtype=torch.int32)) if cu else None)
    for _ in range(3):
        h = up(c["h_in"])
        y, out = m3.mamba3_gated_scan_fwd(**a, h_in=h, h_out=h)
        assert torch.equal(y, got["y"]) and torch.equal(out, got["h_out"])
    if grads:
        got.update(call(c, back))
    worst = {k: R.off(got[k], ref[k]) for k in got}
    note("  " + " ".join(f"{k} {v:.2f}" for k, v in worst.items()))
    assert max(worst.values()) <= 1, worst
