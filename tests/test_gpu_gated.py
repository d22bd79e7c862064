"""The gated linear recurrence on the GPU against its 64-bit form (tests/gated_ref.py): every output within its
type's rounding and the roundings counted along the computation."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
MANY = [0] + sorted(torch.randint(0, 901, (699,), generator=torch.Generator().manual_seed(7)).tolist()) + [900]


def rand(g, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def up(t):
    return t.to(device()) if t is not None else None


def inputs(b, L, D, cu, form, dtype, i, z, state, weight=True, seed=0, memory=0.0):
    """`memory`: how far gates lean to long memories."""
    g = torch.Generator().manual_seed(97 * seed + 13 * L + D)
    S = len(cu) - 1 if cu else b
    w = None
    if form == "decay":
        w = rand(g, D, mean=-4.0 - memory)
    elif weight:
        w = torch.rand(D, generator=g) * 0.9
    return dict(x=rand(g, b, L, D, dtype=dtype), gate=rand(g, b, L, D, dtype=dtype, std=1.5, mean=memory if form == "forget" else 0.0),
                weight=w, form=form, rate=8.0, i=rand(g, b, L, D, dtype=dtype) if i else None,
                z=rand(g, b, L, D, dtype=dtype) if z else None, h_in=rand(g, S, D, std=3.0) if state else None, cu=cu), \
        dict(dy=rand(g, b, L, D, dtype=dtype), dh_out=rand(g, S, D, std=3.0) if state else None)


def call(c, back=None, **more):
    a = {k: up(c[k]) if torch.is_tensor(c[k]) else c[k] for k in ("weight", "form", "rate", "i", "z", "h_in")}
    if c["cu"] is not None:
        a["cu_seqlens"] = up(torch.tensor(c["cu"], dtype=torch.int32))
    w = a.pop("weight")
    if back is None:
        y, h = m3.mamba3_gated_scan_fwd(up(c["x"]), up(c["gate"]), w, **a, **more)
        return dict(y=y, h_out=h)
    return m3.mamba3_gated_scan_bwd(up(c["x"]), up(c["gate"]), w, dy=up(back["dy"]), dh_out=up(back["dh_out"]),
                                    want_dh_in=True, **a, **more)


def check(c, back):
    ref = R.scan(**c, **back)
    got = {**call(c), **call(c, back)}
    want = {"y", "h_out", "dx", "dgate", "dh_in"} | {k for k, n in (("di", "i"), ("dz", "z"), ("dweight", "weight")) if c[n] is not None}
    assert set(got) == want
    worst = {}
    for k in got:
        assert got[k].shape == ref[k][0].shape, k
        assert not got[k].isnan().any(), k
        worst[k] = R.off(got[k], ref[k])
    note("  " + " ".join(f"{k} {v:.2f}" for k, v in worst.items()))
    assert max(worst.values()) <= 1, worst


CASES = [  # batch, seqlen, dim, cu
    (2, 37, 64, None), (1, 1, 8, None), (1, 1, 1, None), (3, 2, 40, None), (1, 33, 1, None), (2, 16, 130, None),
    (1, 65, 129, None), (1, 64, 2, None), (2, 63, 6, None), (1, 90, 72, [0, 0, 1, 3, 3, 40, 41, 90, 90]),
    (1, 34, 9, [0, 17, 17, 34]), (1, 900, 8, MANY), (1, 700, 20, [0, 0, 64, 65, 65, 300, 699, 700]),
    # long enough to run as segments, at their borders and between them
    (1, 128, 34, None), (1, 129, 34, None), (1, 1000, 6, None), (2, 515, 130, None), (3, 384, 7, None),
    (1, 2100, 10, [0, 3, 1100, 2100]), (260, 9, 16, None),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("full", [True, False])
def test_scan(case, form, dtype, full):
    b, L, D, cu = case
    note(f"gated scan b {b} L {L} D {D} packed {cu is not None} {form} {dtype} full {full}")
    check(*inputs(b, L, D, cu, form, dtype, full, full, full, weight=full))


@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("i,z,state", [(True, False, False), (False, True, True), (True, True, False)])
def test_scan_options(form, i, z, state):
    note(f"gated scan options {form} i {i} z {z} state {state}")
    check(*inputs(2, 200, 36, None, form, BF16, i, z, state))
    check(*inputs(1, 260, 15, [0, 100, 101, 260], form, F32, i, z, state))


@pytest.mark.parametrize("form", ["decay", "forget"])
def test_long_memory(form):
    """Decays next to 1, states that live for thousands of tokens over many segments: 1 - a^2 and 1 - a keep
    their relative precision."""
    note(f"gated scan long memory {form}")
    check(*inputs(1, 4000, 4, None, form, F32, True, False, True, weight=form == "decay", memory=6.0))


@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_gates(form, dtype):
    """Gates that close and open entirely, decays of 1 and 0, a rate of zero, weights far out."""
    note(f"gated scan extreme gates {form} {dtype}")
    c, back = inputs(1, 140, 12, None, form, dtype, True, True, True, seed=5)
    for k, v in enumerate((-86.0, 86.0, 300.0, -30.0, 30.0, 0.0)):
        c["gate"][0, 10 + k::7] = v
        c["i"][0, 12 + k::9] = -v
    if form == "decay":
        c["weight"][:6] = torch.tensor([-60.0, -20.0, 10.0, 25.0, 80.0, -9.0])
    else:
        c["weight"][:2] = torch.tensor([0.0, 1.0])
    check(c, back)
    # below the least argument nothing is heard any more
    c["gate"][0, 50] = -1e4
    got = {**call(c), **call(c, back)}
    assert all(bool(v.isfinite().all()) for v in got.values())
    if form == "decay":
        c["rate"] = 0.0
        got = {**call(c), **call(c, back)}
        assert torch.equal(got["h_out"].cpu(), c["h_in"])       # a = 1, u = 0
        assert not got["dx"].any() and not got["dgate"].any() and not got["dweight"].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 33])
def test_views_and_guards(dtype, D):
    """Inputs as parts of wider rows that start at any element; outputs between guards that stay."""
    c, back = inputs(2, 300, D, None, "decay", dtype, True, True, True)
    wide = torch.zeros(2, 300, 5 * D + 3, dtype=dtype)
    parts = {}
    for k, (name, src) in enumerate(dict(x=c["x"], gate=c["gate"], i=c["i"], z=c["z"], dy=back["dy"]).items()):
        wide[:, :, k * D + 1:(k + 1) * D + 1] = src
        parts[name] = k * D + 1
    on = up(wide)
    v = {k: on[:, :, o:o + D] for k, o in parts.items()}
    dense, grads = call(c), call(c, back)
    room = torch.full((2 * 300 * D + 2,), 7.0, dtype=dtype, device=device())
    y, h = m3.mamba3_gated_scan_fwd(v["x"], v["gate"], up(c["weight"]), i=v["i"], z=v["z"], h_in=up(c["h_in"]),
                                    y=room[1:-1].view(2, 300, D))
    assert torch.equal(y, dense["y"]) and torch.equal(h, dense["h_out"])
    assert float(room[0]) == 7.0 and float(room[-1]) == 7.0
    g = m3.mamba3_gated_scan_bwd(v["x"], v["gate"], up(c["weight"]), i=v["i"], z=v["z"], h_in=up(c["h_in"]), dy=v["dy"],
                                 dh_out=up(back["dh_out"]))
    for k in g:
        assert torch.equal(g[k], grads[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,cu", [(50, [3, 10, 10, 41]), (900, [7, 300, 300, 880])])
def test_tokens_outside(dtype, L, cu):
    """Tokens before the first and behind the last sequence, NaN here, take no part, and their rows stay."""
    D = 20
    c, back = inputs(1, L, D, cu, "decay", dtype, True, True, True)
    inside = slice(cu[0], cu[-1])
    for t in (c["x"], c["gate"], c["i"], c["z"], back["dy"]):
        t[:, :cu[0]] = float("nan")
        t[:, cu[-1]:] = float("nan")
    y = torch.full((1, L, D), 5.0, dtype=dtype, device=device())
    call(c, y=y)
    cut = dict(c, cu=[v - cu[0] for v in cu], **{k: c[k][:, inside].contiguous() for k in ("x", "gate", "i", "z")})
    cb = dict(back, dy=back["dy"][:, inside].contiguous())
    ref = R.scan(**cut, **cb)
    assert R.off(y[:, inside], ref["y"]) <= 1
    assert bool((y[:, :cu[0]] == 5).all()) and bool((y[:, cu[-1]:] == 5).all())
    g = call(c, back)
    for k in ("dx", "dgate", "di", "dz"):
        assert R.off(g[k][:, inside], ref[k]) <= 1, k
    for k in ("dweight", "dh_in"):
        assert R.off(g[k], ref[k]) <= 1, k


def test_bad_boundaries():
    """cu_seqlens entries outside the batch are clamped, decreasing ones leave their sequences empty; no access
    lies outside (guards)."""
    L, D = 300, 8
    c, back = inputs(1, L, D, [0, 100, 300], "forget", F32, False, False, False)
    for cu in ([0, 1 << 30, L], [-5, 100, 1 << 20], [0, 200, 100], [250, 20, 300, 7]):
        c["cu"] = cu
        room = torch.full((L * D + 2,), 7.0, device=device())
        y = room[1:-1].view(1, L, D)
        call(c, y=y)
        back["dh_out"] = None
        g = call(c, back)
        assert float(room[0]) == 7.0 and float(room[-1]) == 7.0 and g["dh_in"].shape == (len(cu) - 1, D)
    c["cu"] = [-5, 100, 1 << 20]
    back["dh_out"] = None
    ref = R.scan(**dict(c, cu=[0, 100, 300]), **back)
    got = {**call(c), **call(c, back)}
    for k in ("y", "h_out", "dx", "dgate", "dweight"):
        assert R.off(got[k], ref[k]) <= 1, k


@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 64, 130, 4096])
def test_steps(form, dtype, D):
    """Single tokens through slots from a prompt's state follow the whole sequence; rows without a slot and
    states that no row names stay."""
    note(f"gated steps {form} {dtype} D {D}")
    c, _ = inputs(3, 24, D, None, form, dtype, True, True, True)
    ref = R.scan(**c)
    w = up(c["weight"])
    n = 17
    part = {k: up(c[k][:, :n].contiguous()) for k in ("x", "gate", "i", "z")}
    y, h = m3.mamba3_gated_scan_fwd(part["x"], part["gate"], w, form=form, i=part["i"], z=part["z"], h_in=up(c["h_in"]))
    assert R.off(y, tuple(t[:, :n] for t in ref["y"])) <= 1
    pool = torch.full((7, D), 9.0, device=device())
    slots = torch.tensor([5, -1, 0, 2, 7], dtype=torch.int32, device=device())
    rows = torch.tensor([0, 0, 1, 2, 0])
    pool[[5, 0, 2]] = h
    plain = h.clone()
    for t in range(n, 24):
        wide = torch.cat([c[k][:, t] for k in ("x", "gate", "i", "z")], 1)
        s = {k: up(c[k][:, t][rows].contiguous()) for k in ("x", "gate", "i", "z")}
        yt = torch.full((5, D), 3.0, dtype=dtype, device=device())
        m3.mamba3_gated_step(s["x"], s["gate"], w, h=pool, form=form, i=s["i"], z=s["z"], slots=slots, y=yt)
        assert R.off(yt[[0, 2, 3]], tuple(q[:, t] for q in ref["y"])) <= 1, t
        assert bool((yt[[1, 4]] == 3.0).all())
        # the same without slots, from views of wider rows
        on = up(wide)
        v = [on[:, k * D:(k + 1) * D] for k in range(4)]
        y2 = m3.mamba3_gated_step(v[0], v[1], w, h=plain, form=form, i=v[2], z=v[3])
        assert torch.equal(y2, yt[[0, 2, 3]])
    assert bool((pool[[1, 3, 4, 6]] == 9.0).all()) and torch.equal(pool[[5, 0, 2]], plain)
    assert R.off(plain, ref["h_out"]) <= 1


def test_reproducible_and_in_place():
    """Two runs agree bit for bit; a sequence alone has what it has among others; h_out in h_in's place."""
    c, back = inputs(4, 700, 96, None, "decay", BF16, True, True, True)
    one = {**call(c), **call(c, back)}
    two = {**call(c), **call(c, back)}
    for k in one:
        assert torch.equal(one[k], two[k]), k
    h = up(c["h_in"])
    y, out = m3.mamba3_gated_scan_fwd(up(c["x"]), up(c["gate"]), up(c["weight"]), i=up(c["i"]), z=up(c["z"]), h_in=h, h_out=h)
    assert out.data_ptr() == h.data_ptr() and torch.equal(h, one["h_out"]) and torch.equal(y, one["y"])


# segments whose rows join those before them, a chain over them, one pass, whole; padded and packed
IN_PLACE = [(4, 700, 96, None), (2, 4000, 128, None), (1, 2048, 1024, None), (1, 3000, 512, [0, 1000, 1000, 2900]),
            (1, 30000, 130, None), (1, 1300, 8192, None), (300, 40, 16, None)]


@pytest.mark.parametrize("case", IN_PLACE)
def test_state_in_place(case):
    """h_out in h_in's place has what it has elsewhere, whichever of a sequence's rows ends first."""
    c, _ = inputs(*case, "forget", BF16, True, False, True)
    a = {k: up(c[k]) for k in ("x", "gate", "weight", "i")}
    a.update(form="forget", cu_seqlens=up(torch.tensor(c["cu"], dtype=torch.int32)) if c["cu"] else None)
    h = up(c["h_in"])
    y, out = m3.mamba3_gated_scan_fwd(**a, h_in=h.clone())
    for _ in range(10):
        again = h.clone()
        got, _ = m3.mamba3_gated_scan_fwd(**a, h_in=again, h_out=again)
        assert torch.equal(again, out) and torch.equal(got, y)


def test_empty():
    for b, L, cu in ((0, 9, None), (2, 0, None), (1, 0, [0, 0, 0])):
        c, back = inputs(b, L, 10, cu, "decay", F32, True, True, True)
        got, g = call(c), call(c, back)
        assert torch.equal(got["h_out"].cpu(), c["h_in"]) and torch.equal(g["dh_in"].cpu(), back["dh_out"])
        assert not g["dweight"].any()
        c["h_in"] = back["dh_out"] = None
        got, g = call(c), call(c, back)
        assert not got["h_out"].any() and not g["dh_in"].any()


# few sequences of many channels, long enough for one pass over short runs: several groups of eight runs, sequences that
# end inside, at the end and one token behind a run, more tokens behind the last
PASS = [  # batch, seqlen, dim, cu
    (1, 1300, 8192, None), (1, 2048, 4096, None), (1, 2049, 2050, None), (2, 1100, 2600, None), (3, 700, 4094, None),
    (1, 1200, 8193, None), (1, 2600, 2048, [0, 0, 128, 257, 1400, 1400, 2600]), (1, 2100, 2050, [3, 700, 2095]),
    (8, 1100, 520, None),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", PASS)
@pytest.mark.parametrize("form", ["decay", "forget"])
def test_one_pass(case, form, dtype):
    b, L, D, cu = case
    note(f"gated scan in one pass b {b} L {L} D {D} packed {cu is not None} {form} {dtype}")
    full = form == "decay"
    c, _ = inputs(b, L, D, cu, form, dtype, full, not full, True, memory=2.0)
    ref = R.scan(**c)
    room = torch.full((b * L * D + 2,), 7.0, dtype=dtype, device=device())
    got = call(c, y=room[1:-1].view(b, L, D))
    lo, hi = (cu[0], cu[-1]) if cu else (0, L)
    assert R.off(got["y"][:, lo:hi], tuple(t[:, lo:hi] for t in ref["y"])) <= 1
    assert R.off(got["h_out"], ref["h_out"]) <= 1
    assert bool((got["y"][:, :lo] == 7).all()) and bool((got["y"][:, hi:] == 7).all())
    assert float(room[0]) == 7.0 and float(room[-1]) == 7.0


@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [(1, 1300, 8191, None), (2, 700, 4095, None), (1, 2048, 1023, None), (70, 33, 255, None),
                                  (3, 40, 3, None), (1, 65, 131, None), (1, 1399, 2047, [0, 700, 700, 1399])])
def test_odd_channels(case, form, dtype):
    """An odd count of channels, whose last lane shares one with the lane before it: whole, segments, one pass."""
    c, back = inputs(*case, form, dtype, True, True, True)
    check(c, back)
    if case[0] == 1:
        h = up(c["h_in"])
        a = {k: up(c[k]) for k in ("x", "gate", "weight", "i", "z")}
        a.update(form=form, cu_seqlens=up(torch.tensor(c["cu"], dtype=torch.int32)) if c["cu"] else None)
        y, out = m3.mamba3_gated_scan_fwd(**a, h_in=h.clone())
        got, _ = m3.mamba3_gated_scan_fwd(**a, h_in=h, h_out=h)
        assert torch.equal(got, y) and torch.equal(h, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_pass_many_sequences(dtype):
    """60 packed sequences, some empty, some of one token, a few long ones: more workgroups than whole sequences need."""
    total = 60 * (128 if dtype == F32 else 256) + 20
    cuts = sorted([0, 0, 1, 2, 130, 130, total - 1, total] + [total // 2 + 7 * k for k in range(53)])
    assert len(cuts) == 61
    c, back = inputs(1, total, 1152, cuts, "decay", dtype, True, False, True)
    ref = R.scan(**c, **back)
    got = call(c)
    again = call(c)
    assert all(torch.equal(got[k], again[k]) for k in got)
    assert R.off(got["y"], ref["y"]) <= 1 and R.off(got["h_out"], ref["h_out"]) <= 1


def test_one_pass_repeats():
    """The same bits however the runs are timed: alone, beside other work on another stream, with h_out in h_in's
    place; a workspace of any content."""
    c, _ = inputs(1, 3000, 4096, None, "decay", BF16, True, True, True)
    one = call(c)
    a = {k: up(c[k]) for k in ("x", "gate", "weight", "i", "z", "h_in")}
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device=device())
    for k in range(12):
        with torch.cuda.stream(side):
            for _ in range(k):
                busy = torch.mm(busy, busy) * 1e-3
        ws = torch.full((4 << 20,), (0, 255, 77)[k % 3], dtype=torch.uint8, device=device())
        h = a["h_in"].clone()
        y, out = m3.mamba3_gated_scan_fwd(a["x"], a["gate"], a["weight"], i=a["i"], z=a["z"], h_in=h, h_out=h, workspace=ws)
        assert torch.equal(y, one["y"]) and torch.equal(out, one["h_out"]), k


def test_one_pass_not_finite():
    """Infinities and NaNs, of any bits, stay in their channels and reach the tokens behind them."""
    c, _ = inputs(1, 2100, 4096, None, "forget", F32, False, False, False)
    clean = call(c)
    bad = torch.tensor([-1], dtype=torch.int32).view(F32)        # a NaN of ones
    c["x"][0, 5, 7], c["gate"][0, 600, 9], c["x"][0, 1000, 11] = bad[0], bad[0], float("inf")
    got = call(c)
    hit = [7, 9, 11]
    keep = torch.ones(4096, dtype=torch.bool)
    keep[hit] = False
    assert torch.equal(got["y"][..., keep], clean["y"][..., keep]) and torch.equal(got["h_out"][:, keep], clean["h_out"][:, keep])
    for ch, t in zip(hit, (5, 600, 1000)):
        assert torch.equal(got["y"][0, :t, ch], clean["y"][0, :t, ch]) and not got["y"][0, t:, ch].isfinite().any()
